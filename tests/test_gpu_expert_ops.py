"""The expert-path operators on the GPU against their definitions in 64 bits.

Tolerances are a priori. A rounding to type t costs at most eps(t) / 2 of the
value, and half the smallest subnormal below it. A sum of terms in fp32 whose
longest chain has n additions costs at most n 2^-24 of the sum of the terms'
magnitudes (2^-23 where the tensor core may truncate instead of rounding).
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}


@pytest.fixture(scope="module")
def dfm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mxfp4_routed_expert_top_gb300 as m
    return m


def rounding(dtype):
    return torch.finfo(DT[dtype]).eps / 2


def within(got, want, bound, dtype):
    """|got - want| <= bound + the rounding to dtype (of the value the kernel
    rounded, which lies within bound of want)."""
    got = got.double()
    tol = bound + (want.abs() + bound) * rounding(dtype) + TINY[dtype]
    over = (got - want).abs() - tol
    assert bool((over <= 0).all()), "over by %g at %r" % (over.max().item(), np.unravel_index(over.argmax().item(), over.shape))


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(*shape, g, dtype="f32"):
    return torch.randn(*shape, generator=g, device="cuda").to(DT[dtype])


def random_ids(T, k, E, g, drop=0.0):
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    if drop:
        gone = torch.rand(T, k, generator=g, device="cuda") < drop
        bad = torch.tensor([-1, E, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
        ids = torch.where(gone, bad[torch.randint(0, 4, (T, k), generator=g, device="cuda")], ids)
    return ids.contiguous()


def sorted_places(ids, E):
    """(offs, pos, src) by numpy's stable sort."""
    a = ids.cpu().numpy().reshape(-1)
    valid = (a >= 0) & (a < E)
    order = np.flatnonzero(valid)[np.argsort(a[valid], kind="stable")]
    pos = np.full(a.size, -1, np.int64)
    pos[order] = np.arange(order.size)
    offs = np.concatenate([[0], np.cumsum(np.bincount(a[valid], minlength=E))])
    return offs, pos, order


class Permuted:
    """A permute call's outputs, in buffers filled with a mark first."""

    def __init__(self, dfm, ids, E, x, dtype, H, scales=None, pad=0, stream=None):
        T, k = ids.shape
        A = T * k
        self.rows = torch.full((A, H + pad), 7.0, device="cuda").to(DT[dtype])
        self.offs = torch.full((E + 1,), -7, dtype=torch.int32, device="cuda")
        self.pos = torch.full((A,), -7, dtype=torch.int32, device="cuda")
        self.src = torch.full((A,), -7, dtype=torch.int32, device="cuda")
        kw = {}
        if scales is not None:
            self.rows_scales = torch.full((A, scales.shape[1]), 7.0, device="cuda")
            kw = dict(scales=scales, n_scales=scales.shape[1], rows_scales=self.rows_scales)
        need = dfm.permute_workspace(T, k, E)
        self.workspace = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
        dfm.permute(ids, T, k, E, x, dtype, H, self.rows, self.offs, self.pos, self.src, self.workspace, need,
                    ldx=x.stride(0), ldr=H + pad, stream=stream, **kw)


def check_permuted(r, ids, E, x, H, scales=None, pad=0):
    k = ids.shape[1]
    offs, pos, src = sorted_places(ids, E)
    n = src.size
    assert np.array_equal(r.offs.cpu().numpy(), offs)
    assert np.array_equal(r.pos.cpu().numpy(), pos)
    assert np.array_equal(r.src.cpu().numpy()[:n], src) and bool((r.src[n:] == -7).all())
    token = torch.from_numpy(src // k).cuda()
    byte = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731
    assert torch.equal(byte(r.rows[:n, :H]), byte(x[:, :H])[token])
    mark = byte(torch.full((1, 1), 7.0, device="cuda").to(x.dtype))
    for rest in (r.rows[n:], r.rows[:, H:]):
        if rest.numel():
            assert bool((byte(rest.reshape(-1, 1)) == mark).all())
    if scales is not None:
        assert torch.equal(r.rows_scales[:n], scales[token]) and bool((r.rows_scales[n:] == 7).all())


@pytest.mark.parametrize("T, k, E, H, dtype, drop", [
    (1, 1, 1, 1, "f32", 0), (1, 16, 896, 7168, "bf16", 0), (1, 32, 1024, 63, "f16", 0.3),
    (2, 3, 5, 33, "f16", 0.5), (8, 16, 896, 7168, "bf16", 0.1), (305, 7, 61, 129, "bf16", 0.1),
    (777, 8, 61, 640, "e4m3", 0.1), (777, 8, 3, 641, "e4m3", 0), (65536, 1, 2, 4, "f32", 0.1),
    (4096, 16, 1024, 24, "bf16", 0), (2048, 32, 7, 20, "f32", 0),
    # past one block's counting: counted, summed and placed by chunks
    (65537, 1, 1, 2, "f32", 0), (4099, 17, 1024, 40, "bf16", 0.2), (9000, 32, 999, 7, "f16", 0.05),
    (40000, 32, 33, 16, "e4m3", 0),
])
def test_permute(dfm, T, k, E, H, dtype, drop):
    g = gen(T * k + E)
    ids = random_ids(T, k, E, g, drop)
    x = randn(T, H, g=g, dtype=dtype)
    S = -(-H // 128)
    scales = randn(T, S, g=g) if dtype == "e4m3" else None
    check_permuted(Permuted(dfm, ids, E, x, dtype, H, scales), ids, E, x, H, scales)


@pytest.mark.parametrize("T", [5, 70000])
@pytest.mark.parametrize("what", ["none", "one", "twice"])
def test_permute_all_dropped_one_expert_same_expert_twice(dfm, T, what):
    E, H = 9, 12
    ids = torch.full((T, 2), {"none": -1, "one": 8, "twice": 0}[what], dtype=torch.int32, device="cuda")
    if what == "twice":
        ids[:] = (torch.arange(T, device="cuda") % E)[:, None]
    x = randn(T, H, g=gen(1), dtype="bf16")
    check_permuted(Permuted(dfm, ids, E, x, "bf16", H), ids, E, x, H)


def test_permute_strides_and_odd_addresses(dfm):
    g = gen(2)
    T, k, E, H = 37, 5, 12, 50
    base = torch.zeros(T * k + 1, dtype=torch.int32, device="cuda")
    ids = base[1:].view(T, k)  # 4 bytes past a 16-byte boundary
    ids.copy_(random_ids(T, k, E, g, 0.1))
    wide = randn(T, H + 9, g=g, dtype="bf16")
    for x in (wide, wide[:, 1:]):
        check_permuted(Permuted(dfm, ids, E, x, "bf16", H, pad=3), ids, E, x, H)


@pytest.mark.parametrize("dtype", ["e4m3", "bf16"])
@pytest.mark.parametrize("H", [1, 2, 3, 4, 5, 7, 8, 9, 31, 130])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_permute_rows_off_word_boundaries(dfm, H, dtype, shift):
    """Rows whose every alignment and length modulo a word occurs: no byte
    beside them changes."""
    g = gen(H + shift)
    T, k, E = 23, 3, 4
    ids = random_ids(T, k, E, g, 0.2)
    wide = randn(T, H + 5, g=g, dtype=dtype)
    x = wide.view(torch.uint8 if dtype == "e4m3" else torch.bfloat16)[:, shift:].view(DT[dtype])
    for pad in (0, 1, 2, 3):
        check_permuted(Permuted(dfm, ids, E, x, dtype, H, pad=pad), ids, E, x, H)


def test_permute_empty(dfm):
    offs = torch.full((6,), 9, dtype=torch.int32, device="cuda")
    dfm.permute(None, 0, 2, 5, None, "bf16", 8, None, offs, None, None)
    assert bool((offs == 0).all())


def test_rows_past_32_bits(dfm):
    """More than 2^31 row elements and 2^32 bytes: the last rows are right."""
    T, k, E, H = 20480, 16, 64, 7168
    g = gen(3)
    ids = random_ids(T, k, E, g)
    x = randn(T, H, g=g, dtype="bf16")
    r = Permuted(dfm, ids, E, x, "bf16", H)
    offs, pos, src = sorted_places(ids, E)
    assert T * k * H > 2 ** 31
    assert np.array_equal(r.pos.cpu().numpy(), pos)
    token = torch.from_numpy(src // k).cuda()
    for at in range(0, T * k, T * k // 8):
        assert torch.equal(r.rows[at:at + 512], x[token[at:at + 512]])
    assert torch.equal(r.rows[-512:], x[token[-512:]])
    weights = torch.rand(T, k, generator=g, device="cuda")
    y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    dfm.unpermute(r.rows, "bf16", T * k, r.pos, weights, T, k, H, y)
    # every row of a token is its x: y = x * the sum of its weights
    want = x.double() * weights.double().sum(1, keepdim=True)
    within(y, want, (k + 1) * 2.0 ** -24 * want.abs(), "bf16")


UNPERMUTE_CASES = [
    (1, 1, 1, "f32", 0), (1, 16, 7168, "bf16", 0), (3, 2, 33, "f16", 0.5), (8, 16, 7168, "bf16", 0.2),
    (301, 7, 130, "bf16", 0.1), (129, 32, 2049, "f32", 0.1), (64, 9, 36, "f16", 0), (1200, 3, 64, "f32", 0.9),
    (2, 5, 12, "bf16", 0), (40, 3, 257, "f16", 0.2), (5, 4, 1, "f32", 0), (70, 6, 511, "bf16", 0.1), (33, 2, 20, "f32", 0),
]


def unpermute_inputs(T, k, H, dtype, drop, seed):
    g = gen(seed)
    n = T * k + 3  # three rows that no assignment has
    rows = randn(n, H, g=g, dtype=dtype)
    pos = torch.randperm(n, generator=g, device="cuda")[:T * k].to(torch.int32)
    weights = torch.rand(T, k, generator=g, device="cuda")
    gone = torch.rand(T * k, generator=g, device="cuda") < drop
    if T > 2 and drop:
        gone[:k] = True  # a token without any row
    # dropped as permute marks them, and places behind the rows
    bad = torch.where(torch.rand(T * k, generator=g, device="cuda") < 0.5, -1, n).to(torch.int32)
    pos = torch.where(gone, bad, pos)
    weights.view(-1)[gone] = float("nan")  # a dropped assignment's weight is not read into a sum
    used = torch.zeros(n, dtype=torch.bool, device="cuda")
    used[pos[~gone].long()] = True
    rows[~used] = float("nan")
    return rows, pos, weights, gone.view(T, k), used


@pytest.mark.parametrize("T, k, H, dtype, drop", UNPERMUTE_CASES)
def test_unpermute_and_permute_grad(dfm, T, k, H, dtype, drop):
    rows, pos, weights, gone, _ = unpermute_inputs(T, k, H, dtype, drop, T + H)
    n = rows.shape[0]
    terms = rows[pos.clamp(0, n - 1).long()].double().view(T, k, H).masked_fill(gone[:, :, None], 0)
    w = weights.double().masked_fill(gone, 0)[:, :, None]
    y = torch.full((T, H), 7.0, device="cuda").to(DT[dtype])
    dfm.unpermute(rows, dtype, n, pos, weights, T, k, H, y)
    within(y, (w * terms).sum(1), (k + 1) * 2.0 ** -24 * (w * terms).abs().sum(1), dtype)
    dx = torch.full((T, H), 7.0, device="cuda").to(DT[dtype])
    dfm.permute_grad(rows, dtype, n, pos, T, k, H, dx)
    within(dx, terms.sum(1), k * 2.0 ** -24 * terms.abs().sum(1), dtype)
    if drop and T > 2:
        assert bool((y[0] == 0).all()) and bool((dx[0] == 0).all())


@pytest.mark.parametrize("T, k, H, dtype, drop", UNPERMUTE_CASES)
def test_unpermute_grad(dfm, T, k, H, dtype, drop):
    rows, pos, weights, gone, used = unpermute_inputs(T, k, H, dtype, drop, T + H + 1)
    n = rows.shape[0]
    dy = randn(T, H, g=gen(5), dtype=dtype)
    drows = torch.full((n, H), 7.0, device="cuda").to(DT[dtype])
    dw = torch.full((T, k), 7.0, device="cuda")
    dfm.unpermute_grad(dy, rows, dtype, n, pos, weights, T, k, H, drows, dw)
    assert bool((drows[~used].float() == 7).all())
    place = pos.view(T, k).clamp(0, n - 1).long()
    got = drows[place].double().masked_fill(gone[:, :, None], 0)
    want = (weights.double()[:, :, None] * dy.double()[:, None, :]).masked_fill(gone[:, :, None], 0)
    within(got, want, 2.0 ** -24 * want.abs(), dtype)
    terms = (rows[place].double() * dy.double()[:, None, :]).masked_fill(gone[:, :, None], 0)
    # a thread's own chain (up to 8 columns at a time over 128 threads: at most
    # H / 128 + 8 terms), 5 steps in the warp and 4 over the warps
    chain = -(-H // 128) + 8 + 5 + 4
    within(dw, terms.sum(2), chain * 2.0 ** -24 * terms.abs().sum(2), "f32")
    assert bool((dw[gone] == 0).all())


def test_unpermute_grad_against_differences(dfm):
    """<dy, y(rows + d) - y(rows - d)> / 2 = <drows, d>, and the same for the
    weights: y is linear in each, so central differences have no error but the
    roundings. fp32; n terms a scalar, each with a relative error of at most
    (k + 2) 2^-24 of the magnitudes that enter it."""
    T, k, H = 17, 4, 96
    g = gen(9)
    pos = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32)
    rows, d = randn(T * k, H, g=g), randn(T * k, H, g=g)
    weights, dw_dir = torch.rand(T, k, generator=g, device="cuda"), randn(T, k, g=g)
    dy = randn(T, H, g=g)
    drows, dweights = torch.empty_like(rows), torch.empty_like(weights)
    dfm.unpermute_grad(dy, rows, "f32", T * k, pos, weights, T, k, H, drows, dweights)

    def y(r, w):
        out = torch.empty(T, H, device="cuda")
        dfm.unpermute(r, "f32", T * k, pos, w, T, k, H, out)
        return out.double()

    for plus, minus, inner, size in (
            ((rows + d, weights), (rows - d, weights), (drows.double() * d.double()).sum(), (rows.abs() + d.abs(), weights)),
            ((rows, weights + dw_dir), (rows, weights - dw_dir), (dweights.double() * dw_dir.double()).sum(),
             (rows.abs(), weights + dw_dir.abs()))):
        diff = ((y(*plus) - y(*minus)) * dy.double()).sum() / 2
        magnitude = (y(*size) * dy.abs().double()).sum()
        assert abs(diff - inner).item() <= 2 * (k + 4 + 16) * 2.0 ** -24 * magnitude.item()


# ---- rows in 8 bits -----------------------------------------------------------
def e4m3_nearest(v):
    mag = v.abs()
    e = torch.floor(torch.log2(mag.clamp(min=2.0 ** -20))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return torch.sign(v) * (torch.round(mag / step) * step).clamp(max=448.0)


def quantized(x):
    """codes (fp64 values), scales, and the exact quotients, block by block."""
    x = x.double()
    M, K = x.shape
    codes, scales = torch.empty_like(x), torch.empty(M, -(-K // 128), dtype=torch.float64, device=x.device)
    ratio = torch.empty_like(x)
    for b in range(scales.shape[1]):
        part = x[:, 128 * b:128 * b + 128]
        m = torch.where(part.isfinite(), part.abs(), 0).amax(1, keepdim=True).clamp(min=2.0 ** -100)
        scales[:, b] = (m / 448)[:, 0]
        r = torch.where(part.isfinite(), part * 448 / m, float("nan"))
        ratio[:, 128 * b:128 * b + 128] = r
        codes[:, 128 * b:128 * b + 128] = e4m3_nearest(r)
    return codes, scales, ratio


@pytest.mark.parametrize("M, K, dtype, pad", [
    (1, 1, "f32", 0), (1, 7168, "bf16", 0), (3, 127, "f16", 0), (5, 129, "bf16", 3), (64, 128, "f32", 0),
    (130, 1536, "bf16", 0), (130, 1536, "f16", 8), (77, 1000, "f32", 0), (1000, 264, "bf16", 4), (33, 20, "bf16", 0),
])
def test_quantize(dfm, M, K, dtype, pad):
    g = gen(M + K)
    wide = (torch.randn(M, K + pad, generator=g, device="cuda") *
            torch.exp(3 * torch.randn(M, 1, generator=g, device="cuda"))).to(DT[dtype])
    wide[:, K:] = float("inf")
    wide[0, :min(K, 130)] = 0  # a block of zeros
    x = wide[:, :K]
    codes = torch.full((M, K + pad), 0x55, dtype=torch.uint8, device="cuda")
    nb = -(-K // 128)
    scales = torch.full((M, nb + 1), 7.0, device="cuda")
    dfm.fp8_quantize(wide, dtype, M, K, codes, scales, ldx=K + pad, ldc=K + pad, lds=nb + 1)
    want, s, ratio = quantized(x)
    got = codes[:, :K].contiguous().view(torch.float8_e4m3fn).double()
    if dtype == "f32":
        # the quotient is rounded to fp32 first (twice at most 2^-24): a code
        # may differ where the exact one lies that near to the middle of two
        lower, upper = e4m3_nearest(ratio * (1 - 2.0 ** -22)), e4m3_nearest(ratio * (1 + 2.0 ** -22))
        assert bool(((got == want) | (got == lower) | (got == upper)).all())
    else:
        assert torch.equal(got, want)
    assert torch.equal(scales[:, :nb].double(), s.float().double())
    assert bool((codes[:, K:] == 0x55).all()) and bool((scales[:, nb] == 7).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("K, shift, pad", [(1, 0, 0), (2, 1, 1), (3, 3, 2), (5, 2, 0), (127, 1, 3), (128, 3, 1), (129, 2, 2),
                                           (131, 0, 0), (257, 3, 5), (1001, 1, 0)])
def test_quantize_rows_off_vector_boundaries(dfm, K, shift, pad, dtype):
    """Every alignment of rows of x and codes against each other; NaN beside
    the rows does not enter, and nothing beside the codes is written."""
    g = gen(K + shift)
    M = 13
    wide = torch.randn(M, K + pad + 4, generator=g, device="cuda").to(DT[dtype])
    wide[:, :shift] = float("nan")
    wide[:, shift + K:] = float("nan")
    x = wide[:, shift:shift + K]
    codes = torch.full((M, K + 3), 0x55, dtype=torch.uint8, device="cuda")
    nb = -(-K // 128)
    scales = torch.zeros(M, nb, device="cuda")
    dfm.fp8_quantize(x, dtype, M, K, codes[:, 1:], scales, ldx=wide.shape[1], ldc=K + 3)
    want, s, ratio = quantized(x)
    got = codes[:, 1:K + 1].contiguous().view(torch.float8_e4m3fn).double()
    if dtype == "f32":  # as above: a code may differ next to a middle
        lower, upper = e4m3_nearest(ratio * (1 - 2.0 ** -22)), e4m3_nearest(ratio * (1 + 2.0 ** -22))
        assert bool(((got == want) | (got == lower) | (got == upper)).all())
    else:
        assert torch.equal(got, want)
    assert torch.equal(scales.double(), s.float().double())
    assert bool((codes[:, 0] == 0x55).all()) and bool((codes[:, K + 1:] == 0x55).all())


def test_quantize_infinities_nan_and_extremes(dfm):
    x = torch.zeros(5, 256, device="cuda")
    x[0, 3], x[0, 4], x[0, 130] = float("inf"), 2.0, -float("inf")
    x[1, 0], x[1, 1] = float("nan"), -3.0
    x[2, :128] = torch.finfo(torch.float32).max
    x[2, 5] = 1.0
    x[3, :] = 2.0 ** -120
    x[3, 1] = 1e-45
    x[4, :128] = float("nan")
    codes = torch.empty(5, 256, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(5, 2, device="cuda")
    dfm.fp8_quantize(x, "f32", 5, 256, codes, scales)
    want, s, _ = quantized(x)
    assert torch.equal(torch.nan_to_num(codes.double(), 999.0), torch.nan_to_num(want, 999.0))
    assert torch.equal(scales.double(), s.float().double())
    assert bool(codes[0, 3].isnan()) and bool(codes[0, 130].isnan()) and codes[0, 4].item() == 448
    assert scales[4, 0].item() > 0 and scales[4, 1].item() > 0


# ---- the product ----------------------------------------------------------------
def product_inputs(G, M, N, K, trans, g, pad_code=0x7F):
    """Codes with NaN in the padding, scales; all groups' sizes by the caller."""
    up = lambda n: -(-n // 16) * 16  # noqa: E731

    def codes(*shape):
        v = torch.randn(*shape, generator=g, device="cuda") * 100
        return v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)

    nb, kb = -(-N // 128), -(-K // 128)
    x = codes(M, up(K))
    x[:, K:] = pad_code
    w = codes(G, K, up(N)) if trans else codes(G, N, up(K))
    w[:, :, (N if trans else K):] = pad_code
    xs = torch.exp(torch.randn(M, kb, generator=g, device="cuda")) / 100
    ws = torch.exp(torch.randn(*((G, kb, nb) if trans else (G, nb, kb)), generator=g, device="cuda")) / 1000
    return x, xs, w, ws


def product_definition(x, xs, w, ws, offs, N, K, trans):
    """(y, the sum of the terms' magnitudes), 64 bits."""
    M = x.shape[0]
    dev = x.device
    y, size = (torch.zeros(M, N, dtype=torch.float64, device=dev) for _ in range(2))
    kk, nn = torch.arange(K, device=dev) // 128, torch.arange(N, device=dev) // 128
    value = lambda t: t.view(torch.float8_e4m3fn).double()  # noqa: E731
    for e in range(len(offs) - 1):
        a, b = offs[e], offs[e + 1]
        if a >= b:
            continue
        we, se = (value(w[e]).t(), ws[e].double().t()) if trans else (value(w[e]), ws[e].double())
        we = we[:N, :K] * se[nn][:, kk]
        xe = value(x[a:b, :K].contiguous()) * xs[a:b].double()[:, kk]
        y[a:b], size[a:b] = xe @ we.t(), xe.abs() @ we.abs().t()
    return y, size


def check_product(dfm, counts, N, K, trans, dtype, seed, before=0, after=0, ldy_pad=0, dense=False):
    g = gen(seed)
    offs = np.concatenate([[0], np.cumsum(counts)]) + before
    M, G = int(offs[-1]) + after, len(counts)
    x, xs, w, ws = product_inputs(G, M, N, K, trans, g)
    y = torch.full((M, N + ldy_pad), 7.0, device="cuda").to(DT[dtype])
    o = None if dense else torch.from_numpy(offs.astype(np.int32)).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dfm.fp8_matmul(x, xs, w, ws, o, G, M, N, K, y, dtype, transposed=trans, ldx=x.shape[1], ldw=w.shape[2],
                   ldy=N + ldy_pad, status=status)
    assert status.item() == 0
    want, size = product_definition(x, xs, w, ws, offs.tolist(), N, K, trans)
    a, b = int(offs[0]), int(offs[-1])
    # at most 128 additions in the tensor core and one a block outside it, the
    # scales' product and its use
    chain = 128 + -(-K // 128) + 3
    within(y[a:b, :N], want[a:b], chain * 2.0 ** -23 * size[a:b], dtype)
    for rest in (y[:a], y[b:], y[:, N:]):
        assert bool((rest.float() == 7).all())
    return y


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("counts, N, K, dtype", [
    ([1], 1, 1, "f32"), ([1], 128, 128, "f32"), ([16], 128, 128, "bf16"), ([1], 1536, 7168, "bf16"),
    ([3], 7168, 1536, "f16"), ([0, 5, 0, 0, 17, 1, 0], 130, 300, "f32"), ([1] * 16, 257, 129, "bf16"),
    ([20, 40, 0, 33], 200, 1000, "f32"), ([64, 63, 65], 384, 511, "f32"), ([100, 130, 127, 128, 129], 300, 400, "bf16"),
    ([513, 1, 256, 255], 390, 700, "f32"), ([700], 1000, 260, "f16"), ([256], 128, 4096, "f32"),
    ([2] * 900, 40, 24, "f32"), ([0, 0, 0], 64, 64, "bf16"),
])
def test_product(dfm, counts, N, K, dtype, trans):
    check_product(dfm, counts, N, K, trans, dtype, seed=sum(counts) + N)


@pytest.mark.parametrize("trans", [False, True])
def test_product_rows_outside_the_groups(dfm, trans):
    check_product(dfm, [5, 0, 70, 9], 200, 300, trans, "f32", 4, before=3, after=130, ldy_pad=5)
    check_product(dfm, [1], 130, 300, trans, "bf16", 4, before=300, after=0, ldy_pad=1)


@pytest.mark.parametrize("M", [1, 2, 17, 65, 129, 300])
def test_product_dense(dfm, M):
    check_product(dfm, [M], 500, 900, False, "f32", M, dense=True)


def test_product_offsets_are_clamped(dfm):
    """Offsets outside [0, M] are read as if clamped: nothing else is touched."""
    g = gen(6)
    G, M, N, K = 3, 40, 128, 128
    x, xs, w, ws = product_inputs(G, M, N, K, False, g)
    y = torch.full((M, N), 7.0, device="cuda")
    offs = torch.tensor([-5, 10, 1000, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    dfm.fp8_matmul(x, xs, w, ws, offs, G, M, N, K, y, "f32")
    want, size = product_definition(x, xs, w, ws, [0, 10, 40, 40], N, K, False)
    within(y, want, 132 * 2.0 ** -23 * size, "f32")


@pytest.mark.parametrize("rows", [40, 4000])
def test_product_descending_offsets_write_nothing(dfm, rows):
    g = gen(6)
    G, N, K = 3, 128, 128
    x, xs, w, ws = product_inputs(G, rows, N, K, False, g)
    y = torch.full((rows, N), 7.0, device="cuda")
    offs = torch.tensor([0, 30, 10, 40], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dfm.fp8_matmul(x, xs, w, ws, offs, G, rows, N, K, y, "f32", status=status)
    assert status.item() == 1 and bool((y == 7).all())


def test_product_nan_stays_in_its_row(dfm):
    g = gen(7)
    G, M, N, K = 2, 40, 256, 384
    x, xs, w, ws = product_inputs(G, M, N, K, False, g)
    offs = torch.tensor([0, 21, 40], dtype=torch.int32, device="cuda")
    clean, dirty = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    dfm.fp8_matmul(x, xs, w, ws, offs, G, M, N, K, clean, "f32")
    x[20, 200] = 0x7F
    w[1, 130, 5] = 0xFF
    dfm.fp8_matmul(x, xs, w, ws, offs, G, M, N, K, dirty, "f32")
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[20], bad[21:, 130] = True, True
    assert bool(dirty[bad].isnan().all()) and torch.equal(dirty[~bad], clean[~bad])


def test_product_weights_past_32_bits(dfm):
    """Groups whose weights start beyond 2^32 bytes."""
    G, N, K = 400, 1536, 7168
    assert G * N * K > 2 ** 32
    g = gen(8)
    w = torch.randint(0, 64, (G, N, K), generator=g, device="cuda", dtype=torch.uint8)
    ws = torch.rand(G, N // 128, K // 128, generator=g, device="cuda")
    M = 6
    x, xs, _, _ = product_inputs(1, M, 16, K, False, g)
    offs = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    offs[399], offs[400] = 2, M
    offs[392:399] = 2
    offs[1:392] = 1
    y = torch.empty(M, N, device="cuda")
    dfm.fp8_matmul(x, xs, w, ws, offs, G, M, N, K, y, "f32")
    for e, a, b in ((0, 0, 1), (391, 1, 2), (399, 2, 6)):
        want, size = product_definition(x[a:b], xs[a:b], w[e:e + 1], ws[e:e + 1], [0, b - a], N, K, False)
        within(y[a:b], want, (128 + 56 + 3) * 2.0 ** -23 * size, "f32")


# ---- together, as they are used ---------------------------------------------------
class Experts8:
    """One 8-bit projection per expert between permute and unpermute."""

    def __init__(self, dfm, T, k, E, H, I, seed, drop=0.1):
        g = gen(seed)
        self.dfm, self.dims = dfm, (T, k, E, H, I)
        self.x = randn(T, H, g=g, dtype="bf16")
        self.ids = random_ids(T, k, E, g, drop)
        self.weights = torch.rand(T, k, generator=g, device="cuda")
        _, _, self.w, self.ws = product_inputs(E, 1, I, H, False, g)
        A = T * k
        z = lambda *shape, dtype=torch.float32: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
        self.xq, self.xscale = z(T, H, dtype=torch.uint8), z(T, -(-H // 128))
        self.rows, self.rscale = z(A, H, dtype=torch.uint8), z(A, -(-H // 128))
        self.offs, self.pos, self.src = z(E + 1, dtype=torch.int32), z(A, dtype=torch.int32), z(A, dtype=torch.int32)
        self.h, self.y = z(A, I), z(T, I)
        self.dy = randn(T, I, g=g)
        self.dh, self.dw = z(A, I), z(T, k)
        self.dhq, self.dhscale = z(A, I, dtype=torch.uint8), z(A, -(-I // 128))
        self.drows, self.dx = z(A, H), z(T, H)

    def forward(self, s=None):
        d, (T, k, E, H, I) = self.dfm, self.dims
        A = T * k
        d.fp8_quantize(self.x, "bf16", T, H, self.xq, self.xscale, stream=s)
        d.permute(self.ids, T, k, E, self.xq, "e4m3", H, self.rows, self.offs, self.pos, self.src, scales=self.xscale,
                  n_scales=self.xscale.shape[1], rows_scales=self.rscale, stream=s)
        d.fp8_matmul(self.rows, self.rscale, self.w, self.ws, self.offs, E, A, I, H, self.h, "f32", stream=s)
        d.unpermute(self.h, "f32", A, self.pos, self.weights, T, k, I, self.y, stream=s)

    def backward(self, s=None):
        d, (T, k, E, H, I) = self.dfm, self.dims
        A = T * k
        d.unpermute_grad(self.dy, self.h, "f32", A, self.pos, self.weights, T, k, I, self.dh, self.dw, stream=s)
        d.fp8_quantize(self.dh, "f32", A, I, self.dhq, self.dhscale, stream=s)
        d.fp8_matmul(self.dhq, self.dhscale, self.w, self.ws, self.offs, E, A, H, I, self.drows, "f32",
                     transposed=True, stream=s)
        d.permute_grad(self.drows, "f32", A, self.pos, T, k, H, self.dx, stream=s)

    def outputs(self):
        return [t.clone() for t in (self.y, self.dw, self.dx)]


@pytest.mark.parametrize("T, k, E, H, I", [(1, 4, 8, 256, 128), (50, 4, 8, 256, 384), (600, 2, 5, 512, 272)])
def test_forward_and_backward_together(dfm, T, k, E, H, I):
    """The chain's outputs against the formulas on the values that the codes
    stand for (the 8-bit roundings are the operators' own definition, tested
    above, and are taken from the chain here)."""
    m = Experts8(dfm, T, k, E, H, I, 11)
    m.forward()
    m.backward()
    value = lambda c, s: c.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 1)[:, :c.shape[1]]  # noqa: E731
    w = m.w.view(torch.float8_e4m3fn).double() * m.ws.double().repeat_interleave(128, 1).repeat_interleave(128, 2)[:, :I, :H]
    valid = ((m.ids >= 0) & (m.ids < E))
    e = torch.where(valid, m.ids, 0).long()
    xv = value(m.xq, m.xscale)
    wt = m.weights.double().masked_fill(~valid, 0)
    chain = 128 + -(-max(H, I) // 128) + 3
    h = torch.einsum("th,tkih->tki", xv, w[e])
    hs = torch.einsum("th,tkih->tki", xv.abs(), w[e].abs())
    eps = (chain * 2.0 ** -23 + (k + 2) * 2.0 ** -24)
    within(m.y, (wt[:, :, None] * h).sum(1), eps * (wt[:, :, None] * hs).sum(1), "f32")
    dot = (h * m.dy.double()[:, None]).sum(2).masked_fill(~valid, 0)
    size = (hs * m.dy.double().abs()[:, None]).sum(2).masked_fill(~valid, 0)
    within(m.dw, dot, (chain * 2.0 ** -23 + (-(-I // 256) + 21) * 2.0 ** -24) * size, "f32")
    place = m.pos.view(T, k).clamp(min=0).long()
    dv = value(m.dhq, m.dhscale)[place].masked_fill(~valid[:, :, None], 0)
    within(m.dx, torch.einsum("tki,tkih->th", dv, w[e]), eps * torch.einsum("tki,tkih->th", dv.abs(), w[e].abs()), "f32")
    # the codes of dh stand for weights * dy: an e4m3 rounding each (2^-4 of
    # the value or half the smallest subnormal, 2^-10, of the block's scale)
    dh = (m.weights.double()[:, :, None] * m.dy.double()[:, None, :]).masked_fill(~valid[:, :, None], 0)
    scale = m.dhscale.double().repeat_interleave(128, 1)[:, :I][place].masked_fill(~valid[:, :, None], 0)
    assert bool(((dv - dh).abs() <= dh.abs() * (2.0 ** -4 + 2.0 ** -20) + scale * 2.0 ** -10 * 1.001).all())


def test_same_bits_again_on_other_streams_and_from_a_graph(dfm):
    m = Experts8(dfm, 300, 3, 7, 384, 256, 12)
    m.forward()
    m.backward()
    torch.cuda.synchronize()
    want = m.outputs()

    def wipe():
        for t in (m.y, m.dw, m.dx, m.h, m.drows, m.rows, m.dh):
            t.zero_()
        torch.cuda.synchronize()

    wipe()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        m.forward(s)
        m.backward(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(m.outputs(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        m.forward(s)
        m.backward(s)
    for _ in range(2):
        wipe()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(m.outputs(), want))


def test_two_calls_at_once(dfm):
    """Two sets on two streams with nothing between them: neither sees the other."""
    sets = [Experts8(dfm, 200 + 90 * i, 3, 7, 384, 256, 20 + i) for i in range(2)]
    alone = []
    for m in sets:
        m.forward()
        m.backward()
        torch.cuda.synchronize()
        alone.append(m.outputs())
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(10):
        for m, s in zip(sets, streams):
            m.forward(s)
            m.backward(s)
    torch.cuda.synchronize()
    for m, want in zip(sets, alone):
        assert all(torch.equal(a, b) for a, b in zip(m.outputs(), want))


def test_places_match_the_layers_grouping(dfm):
    """permute's places are those of the layer's own grouping step."""
    T, k, E = 60, 4, 16
    ids = random_ids(T, k, E, gen(30))
    x = randn(T, 8, g=gen(31))
    r = Permuted(dfm, ids, E, x, "f32", 8)
    with dfm.MoE(256, E, k, 64, 0, 0, max_tokens=64) as m:
        offs = torch.zeros(E + 4, dtype=torch.int32, device="cuda")
        tok, slot = (torch.zeros(T * k, dtype=torch.int32, device="cuda") for _ in range(2))
        union = torch.zeros(4, dtype=torch.int32, device="cuda")
        m.step_group(ids, T, offs, tok, slot, union)
        m.sync()
    assert torch.equal(offs[:E + 1], r.offs)
    assert torch.equal(tok * k + slot, r.src)


@pytest.mark.parametrize("T, k, E, H, I", [(300, 3, 7, 384, 256)])
def test_calls_without_a_stream_follow_the_current_one(dfm, T, k, E, H, I):
    """Inside torch.cuda.stream(s), calls that name no stream come after s's own
    work before them and before its work after them. The inputs are zeros until
    that work has written them, so a call that ran early would show."""
    m = Experts8(dfm, T, k, E, H, I, 40)
    m.forward()
    m.backward()
    torch.cuda.synchronize()
    want = m.outputs()
    inputs = [(t, t.clone()) for t in (m.x, m.ids, m.weights, m.dy)]
    for t, _ in inputs:
        t.zero_()
    for t in (m.y, m.dw, m.dx):
        t.fill_(7)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)  # about 10 ms
        for t, value in inputs:
            t.copy_(value)
        m.forward()
        m.backward()
        got = m.outputs()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_calls_without_a_stream_are_captured(dfm):
    m = Experts8(dfm, 100, 3, 7, 384, 256, 41)
    m.forward()
    m.backward()
    torch.cuda.synchronize()
    want = m.outputs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.forward()
        m.backward()
    for t in (m.y, m.dw, m.dx, m.h, m.drows, m.rows, m.dh):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(m.outputs(), want))


# ---- waits that run out -------------------------------------------------------------
def given_up(dfm, role, counts, N, K, trans, seed):
    """(clean y, y, status) of the product where `role` of block 0 gives up."""
    g = gen(seed)
    offs = np.concatenate([[0], np.cumsum(counts)])
    M, G = int(offs[-1]), len(counts)
    x, xs, w, ws = product_inputs(G, M, N, K, trans, g)
    o = torch.from_numpy(offs.astype(np.int32)).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = [torch.full((M, N), 7.0, device="cuda") for _ in range(3)]

    def call(out):
        dfm.fp8_matmul(x, xs, w, ws, o, G, M, N, K, out, "f32", transposed=trans, ldx=x.shape[1], ldw=w.shape[2],
                       status=status)
        torch.cuda.synchronize()
        return status.item()

    assert call(y[0]) == 0
    dfm.test_fp8_give_up(role)
    found = call(y[1])
    status.zero_()
    assert call(y[2]) == 0 and torch.equal(y[2], y[0])  # the request was for one call
    return y[0], y[1], found


GIVE_UP = [  # the 128-row form, few blocks of K and many; more units than SMs; short tiles
    ([300, 200], 300, 200, False), ([300, 200], 300, 1500, True), ([40000], 256, 700, False),
    ([1] * 16, 257, 100, False), ([16] * 340, 120, 1024, True),
]


@pytest.mark.parametrize("role", [1, 2, 3, 4])
@pytest.mark.parametrize("counts, N, K, trans", GIVE_UP)
def test_product_reports_a_wait_that_gave_up(dfm, counts, N, K, trans, role):
    """Status bit 2, NaN in what block 0 computes, every other value as ever."""
    clean, got, status = given_up(dfm, role, counts, N, K, trans, 50)
    assert status == 2
    gone = got.isnan()
    assert bool(gone[0, 0]) and torch.equal(got[~gone], clean[~gone])
    # whole units of at most 128 rows x 256 columns, three of them at most
    assert int(gone.sum()) <= 3 * 128 * 256


@pytest.mark.parametrize("role", [1, 2, 3, 4])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("counts, N, K", [([3], 128, 1024), ([30], 300, 2000), ([1] * 4, 256, 500)])
def test_product_reports_a_wait_that_gave_up_in_a_part_of_k(dfm, counts, N, K, trans, role):
    """Calls whose units are shared by the CTAs of a cluster: what the other
    clusters compute is as ever."""
    clean, got, status = given_up(dfm, role, counts, N, K, trans, 51)
    assert status == 2
    assert torch.equal(got[:, 128:], clean[:, 128:]) and torch.equal(got[counts[0]:], clean[counts[0]:])
    # the sum over the parts is NaN if one of them is
    assert bool(got[:counts[0], :128].isnan().all())


def test_product_give_up_is_checked(dfm):
    for role in (-1, 5):
        with pytest.raises(dfm.DfMoeError):
            dfm.test_fp8_give_up(role)


# ---- scales whose product is no normal number -----------------------------------------
WIDE = [[5, 0, 9], [25, 30], [300, 90], [2] * 300]


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("counts", WIDE)
def test_product_scales_below_the_normal_range(dfm, counts, trans):
    """xs of three sizes (1e-24, quantize's for a row of zeros, ordinary) times
    ws of two: products that are subnormal or below the smallest, whose sums
    are not. Each block of K adds at most half the smallest subnormal to the
    bound; the ordinary rows have the bits that they have alone."""
    g = gen(60)
    M, G, N, K = sum(counts), len(counts), 390, 1200
    x, xs, w, ws = product_inputs(G, M, N, K, trans, g)
    odd = torch.arange(ws.shape[2 if trans else 1], device="cuda") % 2 == 1
    size = torch.where(odd, 2.0 ** -42, 1e-20)
    ws = (0.5 + torch.rand(ws.shape, generator=g, device="cuda")) * (size if trans else size[:, None])
    o = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()

    def call(scales):
        y = torch.full((M, N), 7.0, device="cuda")
        dfm.fp8_matmul(x, scales, w, ws, o, G, M, N, K, y, "f32", transposed=trans, ldx=x.shape[1], ldw=w.shape[2])
        return y

    ordinary = call(xs)
    xs[0::3] *= 1e-22  # from about 1e-2
    xs[1::3] = 2.0 ** -100 / 448
    y = call(xs)
    assert torch.equal(y[2::3], ordinary[2::3])
    want, total = product_definition(x, xs, w, ws, o.tolist(), N, K, trans)
    kb = -(-K // 128)
    within(y, want, (128 + kb + 3) * 2.0 ** -23 * total + kb * 2.0 ** -150, "f32")
    assert bool((y[1, 128:256] != 0).any())


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("counts", WIDE)
def test_product_scales_above_the_normal_range(dfm, counts, trans):
    """xs ws = 2^130 in one block of K: columns whose weights are 0 there get
    nothing from it, and those with x w = 2^-18 get 128 2^-18 2^130 = 2^119."""
    g = gen(61)
    M, G, N, K = sum(counts), len(counts), 300, 640
    x, xs, w, ws = product_inputs(G, M, N, K, trans, g)
    x[:, 128:256] = 1  # the code of 2^-9
    block = (slice(None), slice(128, 256), slice(None)) if trans else (slice(None), slice(None), slice(128, 256))
    w[block] = 0
    w[(slice(None), slice(128, 256), slice(128, N)) if trans else (slice(None), slice(128, N), slice(128, 256))] = 1
    xs[:, 1] = 2.0 ** 70
    if trans:
        ws[:, 1] = 2.0 ** 60
    else:
        ws[:, :, 1] = 2.0 ** 60
    o = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    y = torch.full((M, N), 7.0, device="cuda")
    dfm.fp8_matmul(x, xs, w, ws, o, G, M, N, K, y, "f32", transposed=trans, ldx=x.shape[1], ldw=w.shape[2])
    want, total = product_definition(x, xs, w, ws, o.tolist(), N, K, trans)
    within(y, want, (128 + 5 + 3) * 2.0 ** -23 * total, "f32")
    assert bool((y[:, 128:] == 2.0 ** 119).all())


# ---- behind a kernel that lets its dependents start early ------------------------------
EARLY_KERNEL = r"""
#include <cuda_runtime.h>
#include <stdint.h>
// One warp a block: lets the next kernel's blocks start, waits about 50 us,
// takes all of its SM's tensor memory, gives it back and leaves a mark.
__global__ void early(int* mark) {
  __shared__ uint32_t at;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int i = 0; i < 50; ++i) __nanosleep(1000);
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"((uint32_t)__cvta_generic_to_shared(&at)) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  __syncwarp();
  const uint32_t columns = *(volatile uint32_t*)&at;
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(columns) : "memory");
  if (threadIdx.x == 0) mark[blockIdx.x] = 1;
}
extern "C" __attribute__((visibility("default"))) int launch_early(int* mark, int blocks, void* stream) {
  early<<<blocks, 32, 0, (cudaStream_t)stream>>>(mark);
  return (int)cudaGetLastError();
}
"""


@pytest.fixture(scope="module")
def early_kernel(dfm, tmp_path_factory):
    import ctypes
    import subprocess
    d = tmp_path_factory.mktemp("early")
    (d / "early.cu").write_text(EARLY_KERNEL)
    subprocess.run(["nvcc", "-gencode", "arch=compute_103a,code=sm_103a", "-shared", "-Xcompiler", "-fPIC", "-o",
                    str(d / "early.so"), str(d / "early.cu")], check=True)
    f = ctypes.CDLL(str(d / "early.so")).launch_early
    f.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]
    return f


@pytest.mark.parametrize("counts, N, K", [([1], 1536, 1024), ([5] * 16, 512, 700), ([30] * 9, 512, 700), ([400], 256, 512)])
def test_product_behind_a_kernel_that_takes_tensor_memory_late(dfm, early_kernel, counts, N, K):
    """The product's blocks may start beside that kernel's, one an SM; they
    take no tensor memory before it has ended."""
    g = gen(70)
    M, G = sum(counts), len(counts)
    x, xs, w, ws = product_inputs(G, M, N, K, False, g)
    o = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    mark = torch.zeros(sms, dtype=torch.int32, device="cuda")
    y = [torch.full((M, N), 7.0, device="cuda") for _ in range(2)]
    kw = dict(ldx=x.shape[1], ldw=w.shape[2])
    dfm.fp8_matmul(x, xs, w, ws, o, G, M, N, K, y[0], "f32", **kw)
    torch.cuda.synchronize()
    for _ in range(3):
        assert early_kernel(mark.data_ptr(), sms, None) == 0
        dfm.fp8_matmul(x, xs, w, ws, o, G, M, N, K, y[1], "f32", stream=0, **kw)
    torch.cuda.synchronize()
    assert bool((mark == 1).all()) and torch.equal(y[0], y[1])


# ---- arrays of unaligned rows, to their ends -------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("K", [1, 2, 3, 129, 257])
@pytest.mark.parametrize("M", [1, 2, 3, 5, 40])
def test_quantize_rows_without_gaps_at_odd_addresses(dfm, M, K, dtype):
    """The first and last blocks, whose words of four would reach over x."""
    base = randn(M * K + 8, g=gen(M + K), dtype=dtype)
    for shift in (1, 2, 3):
        x = base[shift:shift + M * K].view(M, K)
        codes = torch.full((M, K), 0x55, dtype=torch.uint8, device="cuda")
        scales = torch.zeros(M, -(-K // 128), device="cuda")
        dfm.fp8_quantize(x, dtype, M, K, codes, scales)
        want, s, ratio = quantized(x)
        got = codes.view(torch.float8_e4m3fn).double()
        lower, upper = e4m3_nearest(ratio * (1 - 2.0 ** -22)), e4m3_nearest(ratio * (1 + 2.0 ** -22))
        assert bool(((got == want) | ((dtype == "f32") & ((got == lower) | (got == upper)))).all())
        assert torch.equal(scales.double(), s.float().double())


@pytest.mark.parametrize("H", [1, 2, 3, 5, 9, 4097])
@pytest.mark.parametrize("T", [1, 2, 700])
def test_permute_rows_without_gaps_at_odd_addresses(dfm, T, H):
    g = gen(T + H)
    k, E = 2, 5
    ids = random_ids(T, k, E, g, 0.1)
    base = torch.randint(0, 255, (T * H + 8,), generator=g, device="cuda", dtype=torch.uint8).view(DT["e4m3"])
    for shift in (0, 1, 2, 3):
        x = base[shift:shift + T * H].view(T, H)
        check_permuted(Permuted(dfm, ids, E, x, "e4m3", H), ids, E, x, H)


@pytest.mark.parametrize("H", [1, 2, 9])
def test_permute_rows_without_gaps_above_one_blocks_counting(dfm, H):
    g = gen(H)
    T, k, E = 33000, 2, 5
    ids = random_ids(T, k, E, g, 0.1)
    base = torch.randint(0, 255, (T * H + 8,), generator=g, device="cuda", dtype=torch.uint8).view(DT["e4m3"])
    x = base[3:3 + T * H].view(T, H)
    check_permuted(Permuted(dfm, ids, E, x, "e4m3", H), ids, E, x, H)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_quantize_next_to_the_middle_of_two_codes(dfm, dtype):
    """Quotients at and next to the middles. bf16 and fp16: the nearest code to
    the exact quotient, ties to even. fp32: also its neighbour, where the
    quotient lies within 2^-23 of its value from the middle."""
    values = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    middle = (values[1:] + values[:-1]) / 2
    g = gen(80)
    m = (1 + torch.rand(64, generator=g, device="cuda")).to(DT[dtype])
    m[:8] = 1.75  # the scale is 2^-8: middles are reached exactly
    x = torch.zeros(64, 3, 128, device="cuda", dtype=DT[dtype])
    near = (middle[None] * m.double()[:, None] / 448).to(DT[dtype])
    ulp = torch.finfo(DT[dtype]).eps
    for i, step in enumerate((0.0, ulp, -ulp)):
        x[:, i, :126] = (near.double() * (1 + step)).to(DT[dtype])
    x[:, :, 127] = m[:, None]
    x = x.view(192, 128)
    codes = torch.empty(192, 128, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(192, 1, device="cuda")
    dfm.fp8_quantize(x, dtype, 192, 128, codes, scales)
    want, s, ratio = quantized(x)
    got = codes.double()
    if dtype == "f32":
        lower, upper = e4m3_nearest(ratio * (1 - 2.0 ** -23)), e4m3_nearest(ratio * (1 + 2.0 ** -23))
        assert bool(((got == want) | (got == lower) | (got == upper)).all())
    else:
        assert torch.equal(got, want)
    assert torch.equal(scales.double(), s.float().double())


# ---- the 128-row form's stores, many units, and what reaches no other value --------------
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("counts, N, K", [([128], 256, 128), ([33, 0, 200], 384, 512), ([300, 129], 1024, 300),
                                          ([65, 190, 1], 640, 1000)])
def test_product_whole_sectors(dfm, counts, N, K, dtype, trans):
    """More than 32 rows a group, rows of y of whole sectors, and columns left
    over behind the last 256."""
    check_product(dfm, counts, N, K, trans, dtype, seed=sum(counts) + K)
    check_product(dfm, counts, N, K, trans, dtype, seed=sum(counts) + K, ldy_pad=16, before=2, after=5)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("counts, N, K", [([700] * 30, 1024, 300), ([257, 0, 1200, 31] * 8, 1300, 1200), ([4000], 2900, 130)])
def test_product_more_units_than_sms(dfm, counts, N, K, dtype, trans):
    """Stages, accumulators and scale buffers carried from unit to unit: 384 to
    720 units of the 128-row form, with 2, 3 and 10 blocks of K."""
    check_product(dfm, counts, N, K, trans, dtype, seed=N + K)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("M, offs, read", [(40, [-5, 10, 1000, 2 ** 31 - 1], [0, 10, 40, 40]),
                                           (90, [-5, 60, 1000, 2 ** 31 - 1], [0, 60, 90, 90]),
                                           (700, [-2 ** 31, -1, 650, 701], [0, 0, 650, 700])])
def test_product_offsets_are_clamped_in_every_form(dfm, M, offs, read, trans):
    g = gen(6)
    G, N, K = 3, 200, 300
    x, xs, w, ws = product_inputs(G, M, N, K, trans, g)
    y = torch.full((M, N), 7.0, device="cuda")
    o = torch.tensor(offs, dtype=torch.int32, device="cuda")
    dfm.fp8_matmul(x, xs, w, ws, o, G, M, N, K, y, "f32", transposed=trans, ldx=x.shape[1], ldw=w.shape[2])
    want, size = product_definition(x, xs, w, ws, read, N, K, trans)
    within(y, want, (128 + 3 + 3) * 2.0 ** -23 * size, "f32")


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("counts", [[9, 7], [21, 19], [200, 150]])
def test_product_nan_stays_in_its_row_in_every_form(dfm, counts, trans):
    g = gen(7)
    G, M, N, K = 2, sum(counts), 256, 384
    x, xs, w, ws = product_inputs(G, M, N, K, trans, g)
    o = torch.tensor([0, counts[0], M], dtype=torch.int32, device="cuda")
    clean, dirty = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    kw = dict(transposed=trans, ldx=x.shape[1], ldw=w.shape[2])
    dfm.fp8_matmul(x, xs, w, ws, o, G, M, N, K, clean, "f32", **kw)
    x[counts[0] - 1, 200] = 0x7F
    xs[3, 1] = float("nan")
    if trans:
        w[1, 5, 130] = 0xFF
    else:
        w[1, 130, 5] = 0xFF
    dfm.fp8_matmul(x, xs, w, ws, o, G, M, N, K, dirty, "f32", **kw)
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[3], bad[counts[0] - 1], bad[counts[0]:, 130] = True, True, True
    assert bool(dirty[bad].isnan().all()) and torch.equal(dirty[~bad], clean[~bad])


# ---- more than one call at once, with nothing left from a call before ---------------------
def chain_outputs(m):
    return (m.xq, m.xscale, m.rows, m.rscale, m.offs, m.pos, m.src, m.h, m.y, m.dh, m.dw, m.dhq, m.dhscale, m.drows, m.dx)


def test_two_chains_at_once_every_round_from_nothing(dfm):
    """Every round starts from wiped buffers and is compared."""
    sets = [Experts8(dfm, 200 + 90 * i, 3, 7, 384, 256, 90 + i) for i in range(2)]
    alone = []
    for m in sets:
        m.forward()
        m.backward()
        torch.cuda.synchronize()
        alone.append(m.outputs())
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(5):
        for i, (m, s) in enumerate(zip(sets, streams)):
            with torch.cuda.stream(s):
                for t in chain_outputs(m):
                    t.zero_()
                m.forward(s)
                m.backward(s)
                got[i].append(m.outputs())
    torch.cuda.synchronize()
    for rounds, want in zip(got, alone):
        for outputs in rounds:
            assert all(torch.equal(a, b) for a, b in zip(outputs, want))


class LargePermute:
    """A permute call above one block's counting, with its own workspace."""

    def __init__(self, dfm, T, seed):
        self.dfm, self.T, self.k, self.E, self.H = dfm, T, 8, 200, 24
        g = gen(seed)
        self.ids = random_ids(T, self.k, self.E, g, 0.1)
        self.x = randn(T, self.H, g=g, dtype="bf16")
        A = T * self.k
        self.rows = torch.zeros(A, self.H, dtype=torch.bfloat16, device="cuda")
        self.offs = torch.zeros(self.E + 1, dtype=torch.int32, device="cuda")
        self.pos, self.src = (torch.zeros(A, dtype=torch.int32, device="cuda") for _ in range(2))
        self.need = dfm.permute_workspace(T, self.k, self.E)
        assert self.need > 0
        self.workspace = torch.zeros(self.need, dtype=torch.uint8, device="cuda")

    def wipe(self):
        for t in (self.rows, self.offs, self.pos, self.src, self.workspace):
            t.zero_()

    def run(self):
        self.dfm.permute(self.ids, self.T, self.k, self.E, self.x, "bf16", self.H, self.rows, self.offs, self.pos,
                         self.src, self.workspace, self.need)

    def right(self):
        offs, pos, src = sorted_places(self.ids, self.E)
        n = src.size
        token = torch.from_numpy(src // self.k).cuda()
        return (np.array_equal(self.offs.cpu().numpy(), offs) and np.array_equal(self.pos.cpu().numpy(), pos)
                and np.array_equal(self.src.cpu().numpy()[:n], src) and torch.equal(self.rows[:n], self.x[token])
                and bool((self.rows[n:] == 0).all()))


def test_permute_with_a_workspace_on_streams_and_from_graphs(dfm):
    """Two calls with workspaces of their own at once; then two captured graphs
    replayed at once."""
    calls = [LargePermute(dfm, 9001, 91), LargePermute(dfm, 20000, 92)]
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(3):
        for c, s in zip(calls, streams):
            with torch.cuda.stream(s):
                c.wipe()
                c.run()
        torch.cuda.synchronize()
        assert all(c.right() for c in calls)
    graphs = []
    for c, s in zip(calls, streams):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            c.run()
    for _ in range(2):
        for c in calls:
            c.wipe()
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        assert all(c.right() for c in calls)
