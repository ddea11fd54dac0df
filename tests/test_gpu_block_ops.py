"""The operators around the routed experts on the GPU against their definitions
in 64 bits.

Tolerances are a priori. U = 2^-24 is half a unit of fp32. A rounding to type t
costs at most eps(t) / 2 of the value, and half the smallest subnormal below it.
A sum in fp32 whose longest chain has n additions costs at most n U of the sum
of the terms' magnitudes (2 n U where the tensor core may truncate instead of
rounding). The library's exponentials, sigmoid and normal distribution function
are within 128 U of values that are not tiny (an exponent's argument of size a is
rounded: a U).
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -126}  # fp32: results that the units flush
U = 2.0 ** -24


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


def randn(*shape, g, dtype="f32", sigma=1.0):
    return (sigma * torch.randn(*shape, generator=g, device="cuda")).to(DT[dtype])


def rows(T, H, g, dtype, pad=0, sigma=1.0, mark=None):
    """[T, H] of a wider array: the padding holds NaN (inputs) or a mark (outputs)."""
    wide = torch.full((T, H + pad), float("nan") if mark is None else mark, device="cuda").to(DT[dtype])
    if mark is None:
        wide[:, :H] = randn(T, H, g=g, dtype=dtype, sigma=sigma)
    return wide[:, :H]


def unmarked(view, mark):
    """The padding behind `view`'s rows is as it was."""
    whole = view._base if view._base is not None else view
    rest = whole[:, view.shape[1]:]
    return bool((rest == torch.tensor(mark).to(rest.dtype)).all()) if rest.numel() else True


def up8(n):
    return -(-n // 8) * 8


# ---- product ----------------------------------------------------------------
def phi(z):
    return 0.5 * torch.special.erfc(-z * math.sqrt(0.5))  # without cancellation: Phi(-10) = 7.62e-24


def act64(z, act, N):
    """act(z), and a bound of |act'| a column of z's."""
    if act == "none":
        return z
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * phi(z)
    return z[:, :N] * torch.sigmoid(z[:, :N]) * z[:, N:]


def slope64(z, act):
    if act == "relu":
        return (z > 0).double()
    if act == "gelu":
        return phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    s = torch.sigmoid(z)
    return s + z * s * (1 - s)


def act_bound(z, bz, act, N):
    """How far act of a z that is bz off is from act(z). |relu'| <= 1, |silu'| and
    |gelu'| < 1.13; evaluating costs 32 U of the value, and of |z| where the
    function is tiny (an exponent's argument is off by U of itself: 100 U)."""
    if act == "none":
        return bz
    if act == "swiglu":
        g, u, bg, bu = z[:, :N], z[:, N:], bz[:, :N], bz[:, N:]
        s = (g * torch.sigmoid(g)).abs()
        bs = 1.13 * bg + 128 * U * s
        return bs * (u.abs() + bu) + s * bu + 2 * U * s * u.abs()
    return 1.13 * bz + 128 * U * act64(z, act, N).abs()


PRODUCTS = [
    # M, N, K, dtype, out, act, bias, residual, pre
    (1, 1, 1, "bf16", "bf16", "none", False, False, False),
    (1, 7168, 2048, "bf16", "bf16", "none", False, True, False),
    (1, 130, 72, "f16", "f32", "gelu", True, True, True),
    (3, 65, 1000, "bf16", "f32", "swiglu", True, True, True),
    (16, 128, 64, "f16", "f16", "relu", True, False, True),
    (17, 200, 8192, "bf16", "bf16", "silu", True, True, False),
    (24, 2048, 7168, "bf16", "bf16", "swiglu", False, False, False),
    (33, 129, 65, "bf16", "f32", "none", True, True, True),
    (64, 64, 4096, "f16", "f32", "swiglu", True, True, True),
    (65, 1, 9, "bf16", "bf16", "gelu", True, True, True),
    (100, 257, 333, "bf16", "f32", "silu", False, True, True),
    (128, 512, 128, "f16", "f16", "none", True, False, False),
    (130, 1030, 777, "f16", "f16", "gelu", True, False, True),
    (200, 333, 640, "bf16", "bf16", "swiglu", True, True, True),
    (513, 640, 1024, "bf16", "f32", "gelu", True, True, True),
    (1024, 1536, 256, "bf16", "bf16", "swiglu", False, True, True),
    (1500, 2052, 520, "f16", "f16", "silu", True, True, True),
    (2049, 2310, 200, "bf16", "f32", "swiglu", True, True, True),
    (2500, 4096, 1031, "bf16", "bf16", "relu", True, True, True),
    (4100, 2048, 96, "f16", "f32", "none", False, False, False),
]


def product_inputs(M, N, K, dtype, act, bias, seed, pad=0):
    g = gen(seed)
    wide = 2 * N if act == "swiglu" else N
    x = rows(M, K, g, dtype, up8(K) - K + pad)
    w = rows(wide, K, g, dtype, up8(K) - K + pad, sigma=1.5 * K ** -0.5)
    b = randn(wide, g=g, dtype=dtype) if bias else None
    return g, wide, x, w, b


def check_product(dfm, M, N, K, dtype, out, act, bias, residual, pre, pad=0, in_place=False, stream=None):
    g, wide, x, w, b = product_inputs(M, N, K, dtype, act, bias, M + N + K, pad)
    r = rows(M, N, g, out, pad % 7) if residual else None
    y = r if in_place else rows(M, N, g, out, (pad + 1) % 5, mark=3.0)
    p = rows(M, wide, g, dtype, (pad + 2) % 5, mark=3.0) if pre else None
    before = r.double().clone() if residual else 0.0
    dfm.matmul(x, w, dtype, M, N, K, y, out, bias=b, act=act, residual=r, pre=p, ldx=x.stride(0), ldw=w.stride(0),
               ldy=y.stride(0), ldr=r.stride(0) if residual else 0, ldp=p.stride(0) if pre else 0, stream=stream)
    xd, wd = x.double(), w.double()
    z = xd @ wd.t()
    bz = 2 * (K + 2) * U * (xd.abs() @ wd.abs().t())
    if bias:
        z = z + b.double()
        bz = bz + U * z.abs()
    if pre:
        within(p, z, bz, dtype)
        assert unmarked(p, 3.0)
    a = act64(z, act, N)
    ba = act_bound(z, bz, act, N)
    want = a + before
    within(y, want, ba + (U * (want.abs() + ba) if residual else 0), out)
    if not in_place:
        assert unmarked(y, 3.0)


@pytest.mark.parametrize("case", PRODUCTS, ids=lambda c: "-".join(map(str, c)))
def test_product(dfm, case):
    check_product(dfm, *case)


@pytest.mark.parametrize("case", [PRODUCTS[2], PRODUCTS[7], PRODUCTS[11], PRODUCTS[15], PRODUCTS[17]],
                         ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("pad", [8, 24])
def test_product_strides(dfm, case, pad):
    """Rows apart: what lies between them is NaN, and is not written in outputs."""
    check_product(dfm, *case, pad=pad)


@pytest.mark.parametrize("case", [PRODUCTS[1], PRODUCTS[10], PRODUCTS[18]], ids=lambda c: "-".join(map(str, c)))
def test_product_adds_to_the_residual_in_place(dfm, case):
    check_product(dfm, *case, in_place=True)


@pytest.mark.parametrize("M", [1, 40, 300, 3000])
def test_product_of_infinities_and_nan_stays_in_its_row(dfm, M):
    N, K = 260, 136
    g, _, x, w, _ = product_inputs(M, N, K, "bf16", "none", False, 5)
    x[M // 2, 7] = float("nan")
    if M > 1:
        x[M - 1, 0] = float("inf")
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    dfm.matmul(x, w, "bf16", M, N, K, y, "bf16", ldx=x.stride(0), ldw=w.stride(0))
    bad = ~torch.isfinite(y.float()).all(1)
    want = torch.zeros(M, dtype=torch.bool, device="cuda")
    want[M // 2] = True
    if M > 1:
        want[M - 1] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("M, N, K, act", [(4, 64, 40000, "none"), (48, 128, 20000, "swiglu"), (100, 200, 33000, "none"), (2100, 1024, 9001, "none"),
                                          (2100, 640, 9001, "swiglu"), (2100, 2050, 7000, "relu"), (5000, 2048, 1600, "none")])
def test_product_sums_keep_their_bits(dfm, M, N, K, act):
    """Of positive terms, so that no error cancels. An addition in tensor memory
    may drop all behind the last bit (2 U): 48 of 16 products each make a part (some
    8 bits of slack for the products of one, aligned to their largest: as much
    again), and the parts are added with U each."""
    g = gen(K)
    x = torch.rand(M, -(-K // 8) * 8, generator=g, device="cuda").to(torch.bfloat16)
    wide = 2 * N if act == "swiglu" else N
    w = torch.rand(wide, -(-K // 8) * 8, generator=g, device="cuda").to(torch.bfloat16)
    y, b = torch.empty(M, N, device="cuda"), None
    if act == "swiglu":  # the gate: 0 but for one column of x, so that silu(1) times the up product's sum is left
        w[:N] = 0
        b = torch.zeros(wide, dtype=torch.bfloat16, device="cuda")
        b[:N] = 1
    dfm.matmul(x, w, "bf16", M, N, K, y, "f32", bias=b, act=act, ldx=x.stride(0), ldw=w.stride(0))
    want = x[:, :K].double() @ w[wide - N:, :K].double().t()
    if act == "swiglu":
        want = want * torch.sigmoid(torch.tensor(1.0, device="cuda", dtype=torch.float64))
    parts = -(-K // 768) + 8
    assert bool(((y.double() - want).abs() <= (4 * 48 + parts + (128 if act == "swiglu" else 0)) * U * want).all())


@pytest.mark.parametrize("case", [
    # M, N, K, dtype, out, act, bias, residual, pre: more than 8192 of k for 16-bit outputs, by tiles of 16, 32 and 64
    # rows and by pairs of 128 and 256 columns, aligned and not, gated and not
    (3, 130, 20000, "bf16", "bf16", "gelu", True, True, True), (40, 96, 9000, "f16", "f16", "swiglu", True, False, True),
    (100, 130, 30000, "bf16", "bf16", "none", False, True, False), (300, 64, 70001, "f16", "f16", "silu", True, True, True),
    (2100, 1024, 9001, "bf16", "bf16", "relu", True, True, True), (2100, 1026, 9001, "f16", "f16", "none", False, False, False),
    (4200, 2304, 8200, "bf16", "bf16", "gelu", True, True, True), (4200, 2306, 8200, "f16", "f16", "none", True, True, True),
    (2100, 640, 17000, "bf16", "bf16", "swiglu", True, True, True), (2100, 1281, 8200, "f16", "f16", "swiglu", False, False, True),
    (4100, 2560, 8264, "bf16", "bf16", "swiglu", True, True, True),
], ids=lambda c: "-".join(map(str, c)))
def test_product_of_many_parts(dfm, case):
    check_product(dfm, *case)


@pytest.mark.parametrize("M, N, K, dtype, out, act", [(2100, 1024, 9001, "bf16", "bf16", "none"), (2100, 1026, 9001, "f16", "f16", "none"),
                                                      (4200, 2304, 8200, "f16", "f16", "none"), (5, 64, 50000, "f16", "f16", "none"),
                                                      (4200, 2306, 16500, "bf16", "bf16", "none"), (100, 40, 262144, "bf16", "f32", "none"),
                                                      (2100, 1280, 20000, "f16", "f16", "swiglu")])
def test_product_of_many_parts_of_positive_terms(dfm, M, N, K, dtype, out, act):
    """No error cancels: 2 U an addition in tensor memory (parts of 8192, or 768, of k, 16
    products at a time and some 8 bits of slack for their alignment: as much again), U a part."""
    g = gen(K)
    x = torch.rand(M, -(-K // 8) * 8, generator=g, device="cuda").to(DT[dtype])
    wide = 2 * N if act == "swiglu" else N
    w = (torch.rand(wide, -(-K // 8) * 8, generator=g, device="cuda") * 2.0 ** -4).to(DT[dtype])
    y, b = torch.empty(M, N, device="cuda", dtype=DT[out]), None
    if act == "swiglu":
        w[:N] = 0
        b = torch.zeros(wide, dtype=DT[dtype], device="cuda")
        b[:N] = 1
    dfm.matmul(x, w, dtype, M, N, K, y, out, bias=b, act=act, ldx=x.stride(0), ldw=w.stride(0))
    want = x[:, :K].double() @ w[wide - N:, :K].double().t()
    if act == "swiglu":
        want = want * torch.sigmoid(torch.tensor(1.0, device="cuda", dtype=torch.float64))
    chunk = 768 if out == "f32" else 8192
    off = (4 * chunk // 16 + -(-K // chunk) + 8 + 128) * U
    within(y, want, off * want, out)


def check_whole_product(dfm, M, N, K, dtype, out, act, bias, residual, pre):
    """check_product with outputs whose rows lie behind each other: whole vectors."""
    g, wide, x, w, b = product_inputs(M, N, K, dtype, act, bias, M + N + 2 * K)
    r = randn(M, N, g=g, dtype=out) if residual else None
    y, p = torch.full((M + 1, N), 3.0, device="cuda").to(DT[out]), torch.full((M + 1, wide), 3.0, device="cuda").to(DT[dtype])
    dfm.matmul(x, w, dtype, M, N, K, y, out, bias=b, act=act, residual=r, pre=p if pre else None, ldx=x.stride(0), ldw=w.stride(0))
    z = x.double() @ w.double().t()
    bz = 2 * (K + 2) * U * (x.double().abs() @ w.double().abs().t())
    if bias:
        z = z + b.double()
        bz = bz + U * z.abs()
    if pre:
        within(p[:M], z, bz, dtype)
    want, bound = act64(z, act, N), act_bound(z, bz, act, N)
    if residual:
        want = want + r.double()
        bound = bound + U * (want.abs() + bound)
    within(y[:M], want, bound, out)
    assert bool((y[M:] == 3).all()) and bool((p[M if pre else 0:] == 3).all())


@pytest.mark.parametrize("out", ["in", "f32"])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("M, N, K, dtype", [(5, 64, 200, "bf16"), (60, 72, 300, "f16"), (200, 96, 520, "bf16"), (2100, 1024, 520, "f16"),
                                            (4100, 2048, 264, "bf16"), (2100, 2560, 1032, "f16")])
def test_product_in_whole_vectors(dfm, M, N, K, dtype, act, out):
    check_whole_product(dfm, M, N, K, dtype, dtype if out == "in" else out, act, True, True, True)


@pytest.mark.parametrize("case", [
    # by tiles of 16, 32 and 64 rows (parts of more than 8192 of k: eight of 8750), by pairs of 128 and 256 columns
    (3, 128, 70000, "bf16", "bf16", "none", False, True, False), (40, 96, 70001, "f16", "f16", "swiglu", True, False, True),
    (300, 64, 70000, "bf16", "bf16", "gelu", True, True, True), (2100, 1024, 9001, "f16", "f16", "gelu", True, True, True),
    (1000, 2560, 8264, "bf16", "bf16", "relu", True, True, True), (1000, 2560, 16500, "f16", "f16", "none", False, False, False),
    (2100, 640, 17000, "f16", "f16", "swiglu", True, True, True), (2100, 1280, 8264, "bf16", "bf16", "swiglu", False, True, False),
], ids=lambda c: "-".join(map(str, c)))
def test_product_of_many_parts_in_whole_vectors(dfm, case):
    check_whole_product(dfm, *case)


@pytest.mark.parametrize("M, N, K, dtype", [(70000, 64, 72, "bf16"), (70001, 61, 130, "f16"), (9000, 2304, 1024, "bf16"), (9001, 1000, 2560, "f16"),
                                            (17000, 2048, 512, "f16")])
def test_product_gradient_of_many_rows_in_16_bits(dfm, M, N, K, dtype):
    """dw of 16 bits, in whole vectors where K is: parts of more than 8192 rows."""
    g, _, x, _, _ = product_inputs(M, N, K, dtype, "none", False, M + N)
    dy = rows(M, N, g, dtype, up8(N) - N, sigma=0.2)
    dw = torch.full((N + 1, K), 3.0, device="cuda").to(DT[dtype])
    dfm.matmul_grad(dy, x, None, dtype, M, N, K, dw=dw, grad_dtype=dtype, lddy=dy.stride(0), ldx=x.stride(0))
    want, size = dy.double().t() @ x.double(), dy.double().abs().t() @ x.double().abs()
    within(dw[:N], want, 2 * (M + 2) * U * size, dtype)
    assert bool((dw[N:] == 3).all())


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "swiglu"])
def test_activations_at_their_ends(dfm, act):
    """Large arguments of either sign: 0 or z, never NaN."""
    z = torch.tensor([-3e4, -120.0, -89.0, -50.0, -10.0, -1.0, -0.0, 0.0, 1e-3, 1.0, 10.0, 50.0, 120.0, 3e4], device="cuda")
    n = z.numel()
    x = torch.zeros(1, 8, dtype=torch.bfloat16, device="cuda")
    x[0, 0] = 1.0
    wide = 2 * n if act == "swiglu" else n
    w = torch.zeros(wide, 8, dtype=torch.bfloat16, device="cuda")
    w[:n, 0] = z.to(torch.bfloat16)
    w[n:, 0] = 1.0
    y = torch.empty(1, n, device="cuda")
    dfm.matmul(x, w, "bf16", 1, n, 8, y, "f32", act=act)
    zd = w[:, 0].double()[None]
    want = act64(zd, act, n)
    # where expf of 88 and more meets a quotient, what is left may be flushed to 0
    assert bool(((y.double() - want).abs() <= 128 * U * want.abs() + 2.0 ** -110).all())


GRADS = [
    # M, N, K, dtype, grad, act
    (1, 1, 1, "bf16", "f32", "none"), (1, 64, 128, "f16", "f16", "gelu"), (5, 3, 7, "bf16", "bf16", "swiglu"),
    (16, 130, 72, "bf16", "f32", "silu"), (33, 257, 65, "f16", "f32", "swiglu"), (64, 64, 64, "bf16", "f32", "relu"),
    (65, 100, 200, "f16", "f16", "none"), (129, 512, 130, "bf16", "bf16", "gelu"), (1001, 1030, 777, "f16", "f16", "gelu"),
    (700, 192, 2310, "bf16", "f32", "swiglu"), (2100, 1280, 1100, "bf16", "bf16", "swiglu"),
    (3000, 77, 2050, "f16", "f32", "none"), (520, 2304, 2304, "bf16", "f32", "none"), (5000, 40, 24, "bf16", "f32", "silu"),
]


def check_gradient(dfm, M, N, K, dtype, grad, act, wanted=("dx", "dw", "dbias"), pad=0):
    g, wide, x, w, _ = product_inputs(M, N, K, dtype, act, False, M + 3 * N + K, pad)
    dy = rows(M, N, g, dtype, up8(N) - N + pad, sigma=0.2)
    z = rows(M, wide, g, dtype, pad % 3, sigma=1.5) if act != "none" else None
    dz = rows(M, wide, g, dtype, up8(wide) - wide + pad, mark=3.0) if act != "none" else None
    out = {"dx": rows(M, K, g, dtype, pad % 5, mark=3.0), "dw": rows(wide, K, g, grad, (pad + 1) % 5, mark=3.0),
           "dbias": torch.full((wide,), 3.0, device="cuda").to(DT[grad])}
    kw = {key: out[key] for key in wanted}
    if act != "none":
        kw.update(pre=z, dz=dz, ldp=z.stride(0), lddz=dz.stride(0))
    dfm.matmul_grad(dy, x, w, dtype, M, N, K, grad_dtype=grad, act=act, lddy=dy.stride(0), ldx=x.stride(0), ldw=w.stride(0),
                    lddx=out["dx"].stride(0), lddw=out["dw"].stride(0), **kw)
    dyd = dy.double()
    if act == "none":
        want, off = dyd, torch.zeros_like(dyd)
        sums_off = off
    else:
        zd = z.double()
        if act == "swiglu":
            gate, u = zd[:, :N], zd[:, N:]
            want = torch.cat([dyd * u * slope64(gate, act), dyd * gate * torch.sigmoid(gate)], 1)
            # the slope is s + g s (1 - s): its parts cancel near its zero
            most = torch.cat([(dyd * u).abs() * (torch.sigmoid(gate) * (1 + gate.abs())), want[:, N:].abs()], 1)
        else:
            want = dyd * slope64(zd, act)
            most = dyd.abs() * (1 + zd.abs())
        sums_off = 128 * U * most
        within(dz, want, sums_off, dtype)
        assert unmarked(dz, 3.0)
        off = sums_off + (want.abs() + sums_off) * rounding(dtype) + TINY[dtype]
    size = want.abs() + off
    for key in out:
        if key not in wanted:
            assert bool((out[key] == 3).all())
    if "dx" in wanted:
        within(out["dx"], want @ w.double(), off @ w.double().abs() + 2 * (wide + 2) * U * (size @ w.double().abs()), dtype)
        assert unmarked(out["dx"], 3.0)
    if "dw" in wanted:
        within(out["dw"], want.t() @ x.double(), off.t() @ x.double().abs() + 2 * (M + 2) * U * (size.t() @ x.double().abs()), grad)
        assert unmarked(out["dw"], 3.0)
    if "dbias" in wanted:
        within(out["dbias"], want.sum(0), sums_off.sum(0) + (M + 2) * U * size.sum(0), grad)


@pytest.mark.parametrize("case", GRADS, ids=lambda c: "-".join(map(str, c)))
def test_product_gradient(dfm, case):
    check_gradient(dfm, *case)


@pytest.mark.parametrize("case", [(9000, 130, 72, "bf16", "bf16", "none"), (20000, 64, 200, "f16", "f16", "gelu"), (9001, 1024, 1100, "bf16", "bf16", "none"),
                                  (8500, 1030, 1101, "f16", "f16", "silu"), (9000, 2304, 2304, "bf16", "bf16", "none"), (8300, 300, 264, "bf16", "bf16", "swiglu")],
                         ids=lambda c: "-".join(map(str, c)))
def test_product_gradient_of_many_rows(dfm, case):
    """dw's k is the rows: more than 8192 of them, in 16 bits."""
    check_gradient(dfm, *case)


@pytest.mark.parametrize("wanted", [("dx",), ("dw",), ("dbias",), ("dx", "dbias"), ("dw", "dbias"), ()])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_product_gradient_of_some(dfm, act, wanted):
    if wanted or act != "none":
        check_gradient(dfm, 77, 136, 96, "bf16", "f32", act, wanted, pad=8)


def test_product_gradient_of_no_rows_is_zero(dfm):
    dw, db = rows(6, 5, None, "f32", 3, mark=3.0), torch.full((6,), 3.0, device="cuda")
    dfm.matmul_grad(None, None, None, "bf16", 0, 3, 5, dw=dw, dbias=db, act="swiglu", ldx=8, lddw=8, lddz=8)
    assert bool((dw == 0).all()) and bool((db == 0).all()) and unmarked(dw, 3.0)


@pytest.mark.parametrize("M, N, K", [(9000, 64, 2048), (64, 5000, 2048), (700, 200, 2048)])
def test_what_follows_a_product_gradient_finds_both(dfm, M, N, K):
    """dx and dw run side by side; a kernel behind them reads either whole, also
    from a graph."""
    g, _, x, w, _ = product_inputs(M, N, K, "bf16", "none", False, 17)
    dy = randn(M, N, g=g, dtype="bf16")
    dx, n = (torch.zeros(M, K, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dw, m = (torch.zeros(N, K, device="cuda") for _ in range(2))  # fp32, as dw is by default

    def run():
        dx.zero_()
        dw.zero_()
        dfm.matmul_grad(dy, x, w, "bf16", M, N, K, dx=dx, dw=dw)
        dfm.block_norm(None, dx, "bf16", M, K, n=n)
        dfm.block_norm(None, dw, "f32", N, K, n=m)
    dfm.matmul_grad(dy, x, w, "bf16", M, N, K, dx=dx, dw=dw)
    torch.cuda.synchronize()
    want = torch.empty_like(n), torch.empty_like(m)
    dfm.block_norm(None, dx, "bf16", M, K, n=want[0])
    dfm.block_norm(None, dw, "f32", N, K, n=want[1])
    torch.cuda.synchronize()
    for _ in range(5):
        run()
        assert torch.equal(n, want[0]) and torch.equal(m, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(5):
        n.zero_()
        m.zero_()
        graph.replay()
        assert torch.equal(n, want[0]) and torch.equal(m, want[1])


def test_product_gradient_against_differences(dfm):
    """<dx, d> is how the loss <dy, y> moves along d: central differences of the
    definition in 64 bits."""
    M, N, K = 9, 40, 24
    g, wide, x, w, b = product_inputs(M, N, K, "f16", "swiglu", True, 3)
    dy = randn(M, N, g=g, dtype="f16")
    pre = torch.empty(M, wide, dtype=torch.float16, device="cuda")
    y = torch.empty(M, N, device="cuda")
    dfm.matmul(x, w, "f16", M, N, K, y, "f32", bias=b, act="swiglu", pre=pre)
    dx, dw = torch.empty_like(x), torch.empty(wide, K, device="cuda")
    db, dz = torch.empty(wide, device="cuda"), torch.empty(M, wide, dtype=torch.float16, device="cuda")
    dfm.matmul_grad(dy, x, w, "f16", M, N, K, dx=dx, dw=dw, dbias=db, act="swiglu", pre=pre, dz=dz)

    def loss(x, w, b):
        return (act64(x @ w.t() + b, "swiglu", N) * dy.double()).sum().item()
    at = [x.double(), w.double(), b.double()]
    for i, grad in enumerate((dx, dw, db)):
        d = torch.randn(grad.shape, generator=g, device="cuda", dtype=torch.float64)
        moved = [[v + s * 1e-5 * d if j == i else v for j, v in enumerate(at)] for s in (1, -1)]
        slope = (loss(*moved[0]) - loss(*moved[1])) / 2e-5
        # z and dz are rounded to fp16 (2^-11 each): as many errors of that size as dz has
        # elements, adding up at worst
        terms = dz.double().abs()
        size = (terms @ at[1].abs() if i == 0 else terms.t() @ at[0].abs() if i == 1 else terms.sum(0)) * d.abs()
        size = size.sum().item()
        assert abs((grad.double() * d).sum().item() - slope) <= 8 * 2.0 ** -11 * size


@pytest.mark.parametrize("M, N, K", [(4, 256, 512), (300, 256, 512), (3000, 2304, 512)])
@pytest.mark.parametrize("role", [1, 2, 3])
def test_product_whose_wait_runs_out_says_so(dfm, M, N, K, role):
    """NaN and the status bit for the block that gave up; the next call is clean."""
    g, _, x, w, _ = product_inputs(M, N, K, "bf16", "none", False, 9)
    y = torch.zeros(M, N, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dfm.test_matmul_give_up(role)
    dfm.matmul(x, w, "bf16", M, N, K, y, "f32", status=status)
    assert status.item() == 2 and bool(torch.isnan(y).any())
    good = ~torch.isnan(y)
    status.zero_()
    again = torch.zeros(M, N, device="cuda")
    dfm.matmul(x, w, "bf16", M, N, K, again, "f32", status=status)
    assert status.item() == 0 and bool(torch.isfinite(again).all())
    assert torch.equal(y[good], again[good])


@pytest.mark.parametrize("M, N, K, out", [(4, 256, 20000, "f32"), (300, 256, 20000, "f32"), (3000, 2304, 2500, "f32"), (3000, 2050, 2500, "f32"),
                                          (3000, 512, 30000, "bf16")])
@pytest.mark.parametrize("role", [1, 2, 3])
def test_product_of_many_parts_whose_wait_runs_out_says_so(dfm, M, N, K, out, role):
    g, _, x, w, _ = product_inputs(M, N, K, "bf16", "none", False, 9)
    y, again = (torch.zeros(M, N, device="cuda", dtype=DT[out]) for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dfm.test_matmul_give_up(role)
    dfm.matmul(x, w, "bf16", M, N, K, y, out, status=status, ldx=x.stride(0), ldw=w.stride(0))
    assert status.item() == 2 and bool(torch.isnan(y).any())
    good = ~torch.isnan(y)
    status.zero_()
    dfm.matmul(x, w, "bf16", M, N, K, again, out, status=status, ldx=x.stride(0), ldw=w.stride(0))
    assert status.item() == 0 and bool(torch.isfinite(again).all())
    assert torch.equal(y[good], again[good])


def test_product_rows_past_32_bits(dfm):
    """More than 2^31 elements of y, and of x."""
    M, N, K = 300_000, 8192, 8
    g, _, x, w, _ = product_inputs(M, N, K, "bf16", "none", False, 1)
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    dfm.matmul(x, w, "bf16", M, N, K, y, "bf16")
    for at in (0, 150_001, M - 64):
        part = x[at:at + 64].double()
        within(y[at:at + 64], part @ w.double().t(), 20 * U * (part.abs() @ w.double().abs().t()), "bf16")
    wide = torch.empty(1, device="cuda")
    del y, wide
    M, K, ld = 70_000, 64, 40_000
    base = torch.zeros(M * ld, dtype=torch.bfloat16, device="cuda")
    x = base.view(M, ld)[:, :K]
    x[-3:] = randn(3, K, g=g, dtype="bf16")
    w = randn(32, K, g=g, dtype="bf16")
    y = torch.empty(M, 32, device="cuda")
    dfm.matmul(x, w, "bf16", M, 32, K, y, "f32", ldx=ld)
    assert bool((y[:-3] == 0).all())
    within(y[-3:], x[-3:].double() @ w.double().t(), 2 * 66 * U * (x[-3:].double().abs() @ w.double().abs().t()), "f32")


# ---- norms ------------------------------------------------------------------
EPS = 1e-6


def rms64(v):
    return torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)


def gate64(gate, kind):
    return 1.0 if gate is None else gate.double()[:, None] if kind == "token" else gate.double()


def make_gate(kind, T, H, dtype, wtype, g, pad=0):
    if kind == "none":
        return None
    if kind == "channel":
        return randn(H, g=g, dtype=wtype)
    return randn(T, g=g) if kind == "token" else rows(T, H, g, dtype, pad)


def forward64(u, r, post, q, gate, kind, scale, v):
    a = u
    if post:
        a = u * rms64(u) * (1.0 if q is None else q.double())
    h = gate64(gate, kind) * a if a is not None else 0.0
    if r is not None:
        h = h + scale * r
    return a, h, h * rms64(h) * (1.0 if v is None else v.double())


NORMS = [
    # T, H, dtype, weights, post, gate, scale
    (1, 1, "f32", "f32", True, "none", 1.0), (1, 7168, "bf16", "bf16", True, "none", 1.0), (3, 8, "f16", "f32", True, "channel", 0.5),
    (5, 33, "bf16", "f32", True, "token", 1.0), (2, 256, "f16", "f16", True, "full", -1.5), (7, 257, "f32", "f32", False, "channel", 1.0),
    (40, 512, "bf16", "bf16", True, "channel", 1.0), (9, 520, "f32", "f32", True, "full", 1.0), (17, 1023, "f16", "f32", False, "token", 2.0),
    (6, 2049, "f32", "f32", True, "token", 1.0), (4, 4096, "bf16", "f32", False, "none", 1.0), (301, 1536, "f16", "f16", True, "full", 1.0),
    (1, 8192, "f32", "f32", True, "channel", 1.0), (3, 8200, "bf16", "bf16", True, "channel", 1.0), (2, 16384, "bf16", "f32", True, "full", 1.0),
    (2, 16385, "f16", "f32", True, "channel", 1.0), (3, 32768, "bf16", "f32", True, "channel", 1.0), (1, 32767, "f32", "f32", True, "token", 1.0),
    (700, 128, "bf16", "f32", True, "channel", 1.0), (2000, 72, "f32", "f32", True, "token", 0.5), (1100, 3584, "bf16", "bf16", True, "channel", 1.0),
]


def check_norm(dfm, T, H, dtype, wtype, post, kind, scale, pad=0, weights=True):
    g = gen(T + H)
    u, r = rows(T, H, g, dtype, pad), rows(T, H, g, dtype, pad, sigma=3.0)
    q = randn(H, g=g, dtype=wtype) if post and weights else None
    v = randn(H, g=g, dtype=wtype) if weights else None
    gate = make_gate(kind, T, H, dtype, wtype, g, pad)
    h, n = rows(T, H, g, dtype, pad, mark=3.0), rows(T, H, g, dtype, 2 * pad, mark=3.0)
    dfm.block_norm(u, r, dtype, T, H, h, n, post=post, post_weight=q, gate=gate, gate_kind=kind, residual_scale=scale,
                   pre_weight=v, weight_dtype=wtype, eps=EPS, ldu=u.stride(0), ldr=r.stride(0), ldh=h.stride(0),
                   ldn=n.stride(0), ldg=gate.stride(0) if kind == "full" else 0)
    a, want_h, want_n = forward64(u.double(), r.double(), post, q, gate, kind, scale, v)
    # a mean of squares has chains of at most 32 + 10 additions and two roundings a term: its root is off by 23 U
    part = (gate64(gate, kind) * a).abs()
    bound = 32 * U * part + U * (abs(scale) * r.double().abs() + want_h.abs())
    within(h, want_h, bound, dtype)
    rel = (bound.pow(2).sum(1, keepdim=True) / want_h.pow(2).sum(1, keepdim=True)).sqrt()  # Cauchy: how far h's root may be off
    vv = 1.0 if v is None else v.double().abs()
    within(n, want_n, vv * rms64(want_h) * bound * (1 + rel) + (32 * U + rel) * want_n.abs(), dtype)
    assert unmarked(h, 3.0) and unmarked(n, 3.0)


@pytest.mark.parametrize("case", NORMS, ids=lambda c: "-".join(map(str, c)))
def test_norm(dfm, case):
    check_norm(dfm, *case)


@pytest.mark.parametrize("case", [NORMS[2], NORMS[4], NORMS[7], NORMS[11]], ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("pad", [3, 8])
def test_norm_strides(dfm, case, pad):
    check_norm(dfm, *case, pad=pad)


def test_norm_without_weights(dfm):
    check_norm(dfm, 37, 640, "bf16", "f32", True, "token", 1.0, weights=False)


@pytest.mark.parametrize("H", [24, 77, 1024, 7168])
def test_norm_of_the_residual_alone_is_the_stacks(dfm, H):
    """Without u and weights: x / sqrt(mean x^2 + eps), as the stack's layers take it."""
    T = 5
    x = rows(T, H, gen(H), "bf16")
    n = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    dfm.block_norm(None, x, "bf16", T, H, n=n, eps=EPS)
    want = x.double() * rms64(x.double())
    within(n, want, 32 * U * want.abs(), "bf16")


@pytest.mark.parametrize("H", [64, 100, 4096])
def test_norm_parts(dfm, H):
    """Only h, only n, no residual; outputs in place of the inputs."""
    T, g = 11, gen(H)
    u, r, q, v = rows(T, H, g, "f32"), rows(T, H, g, "f32"), randn(H, g=g), randn(H, g=g)
    h, n = torch.empty(T, H, device="cuda"), torch.empty(T, H, device="cuda")
    kw = dict(post=True, post_weight=q, pre_weight=v)
    dfm.block_norm(u, r, "f32", T, H, h, n, **kw)
    only = torch.empty(T, H, device="cuda")
    dfm.block_norm(u, r, "f32", T, H, h=only, **kw)
    assert torch.equal(only, h)
    dfm.block_norm(u, r, "f32", T, H, n=only, **kw)
    assert torch.equal(only, n)
    dfm.block_norm(u, None, "f32", T, H, h=only, post=True, post_weight=q)
    want = u.double() * rms64(u.double()) * q.double()
    within(only, want, 32 * U * want.abs(), "f32")
    u2, r2 = u.clone(), r.clone()
    dfm.block_norm(u2, r2, "f32", T, H, h=r2, n=u2, **kw)
    assert torch.equal(r2, h) and torch.equal(u2, n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H", [48, 1000, 8192])
def test_norm_of_huge_tiny_and_broken_rows(dfm, dtype, H):
    g = gen(H)
    size = torch.tensor([1e30, 1e-30, 0.0, 1e18, 1e20, 3e37], device="cuda")[:, None]
    T = 8
    x = torch.zeros(T, H, device="cuda")
    x[:6] = size * torch.randn(6, H, generator=g, device="cuda").clamp(-4, 4)
    x[6:] = torch.randn(2, H, generator=g, device="cuda")
    x[6, H // 2] = float("nan")
    x[7, 0] = float("inf")
    x = x.to(DT[dtype])
    n, h = torch.empty_like(x), torch.empty_like(x)
    dfm.block_norm(x, None, dtype, T, H, h, n, post=True, eps=EPS)
    want = x[:6].double() * rms64(x[:6].double())
    within(h[:6], want, 64 * U * want.abs(), dtype)
    assert bool(torch.isnan(h[6].float()).all())
    # next to an infinity nothing is left of the others
    assert bool(torch.isnan(h[7, 0].float())) and bool((h[7, 1:] == 0).all())
    dn, dx = torch.randn(T, H, generator=g, device="cuda").to(DT[dtype]), torch.empty_like(x)
    dfm.block_norm_grad(None, dn, None, x, dtype, T, H, dresidual=dx, eps=EPS)
    xd, dd = x[:6].double(), dn[:6].double()
    rms = rms64(xd)
    hat = xd * rms
    along = (dd * hat).mean(1, keepdim=True)
    want = rms * (dd - hat * along)
    bound = rms * (128 + math.ceil(H / 256)) * U * (dd.abs() + hat.abs() * (dd * hat).abs().mean(1, keepdim=True))
    within(dx[:6], want, bound, dtype)


def grad64(dh, dn, u, h, post, q, gate, kind, scale, v):
    """The gradients, and for each the sum of its terms' magnitudes."""
    H = h.shape[1]
    G, mag = torch.zeros_like(h), torch.zeros_like(h)
    out = {}
    if dh is not None:
        G, mag = G + dh, mag + dh.abs()
    if dn is not None:
        y = dn * (1.0 if v is None else v.double())
        rms = rms64(h)
        hat = h * rms
        G = G + rms * (y - hat * (y * hat).mean(1, keepdim=True))
        mag = mag + rms * (y.abs() + hat.abs() * (y * hat).abs().mean(1, keepdim=True))
        out["dpre_weight"] = (dn * hat).sum(0), (dn * hat).abs().sum(0)
    out["dresidual"] = scale * G, abs(scale) * mag
    if u is None:
        return out
    gt = gate64(gate, kind)
    da, dam = gt * G, abs(gt) * mag if kind != "none" else mag
    a = u
    if post:
        rms = rms64(u)
        hat = u * rms
        qq = 1.0 if q is None else q.double()
        a = hat * qq
        y, ym = da * qq, dam * abs(qq)
        out["dpost_weight"] = (da * hat).sum(0), (dam * hat.abs()).sum(0)
        out["du"] = rms * (y - hat * (y * hat).mean(1, keepdim=True)), rms * (ym + hat.abs() * (ym * hat.abs()).mean(1, keepdim=True))
    else:
        out["du"] = da, dam
    each, em = G * a, mag * a.abs()
    out["dgate"] = {"channel": (each.sum(0), em.sum(0)), "token": (each.sum(1), em.sum(1)), "full": (each, em), "none": None}[kind]
    return out


def check_norm_grad(dfm, T, H, dtype, wtype, post, kind, scale, pad=0, weights=True, dh_too=True, dn_too=True, wanted=None):
    g = gen(T + 7 * H)
    u, h = rows(T, H, g, dtype, pad), rows(T, H, g, dtype, pad, sigma=2.0)
    dh = rows(T, H, g, dtype, pad, sigma=0.3) if dh_too else None
    dn = rows(T, H, g, dtype, pad, sigma=0.3) if dn_too else None
    q = randn(H, g=g, dtype=wtype) if post and weights else None
    v = randn(H, g=g, dtype=wtype) if weights and dn_too else None
    gate = make_gate(kind, T, H, dtype, wtype, g, pad)
    out = {"du": rows(T, H, g, dtype, pad, mark=3.0), "dresidual": rows(T, H, g, dtype, 2 * pad, mark=3.0)}
    if post:
        out["dpost_weight"] = torch.full((H,), 3.0, device="cuda")
    if dn_too:
        out["dpre_weight"] = torch.full((H,), 3.0, device="cuda")
    if kind != "none":
        out["dgate"] = {"channel": lambda: torch.full((H,), 3.0, device="cuda"), "token": lambda: torch.full((T,), 3.0, device="cuda"),
                        "full": lambda: rows(T, H, g, dtype, pad, mark=3.0)}[kind]()
    if wanted is not None:
        out = {key: o for key, o in out.items() if key in wanted}
    size = dfm.block_norm_grad_workspace(T, H)
    workspace = torch.empty(size, dtype=torch.uint8, device="cuda")
    lds = dict(lddu="du", lddr="dresidual")
    if kind == "full":
        lds["lddg"] = "dgate"
    dfm.block_norm_grad(dh, dn, u, h, dtype, T, H, post=post, post_weight=q, gate=gate, gate_kind=kind, residual_scale=scale,
                        pre_weight=v, weight_dtype=wtype, eps=EPS, workspace=workspace, workspace_bytes=size,
                        lddh=dh.stride(0) if dh_too else 0, lddn=dn.stride(0) if dn_too else 0, ldu=u.stride(0),
                        ldh=h.stride(0), ldg=gate.stride(0) if kind == "full" else 0,
                        **{key: out[o].stride(0) for key, o in lds.items() if o in out}, **out)
    want = grad64(dh.double() if dh_too else None, dn.double() if dn_too else None, u.double(), h.double(), post, q, gate, kind, scale, v)
    # A row's sums have chains of at most 32 + 10 additions, and a value takes the sums, the roots (23 U) and some
    # twenty roundings: 128 U of the terms' magnitudes for one norm, twice that for both. Column sums add T terms in
    # chains that are no longer than T + 64.
    for key, o in out.items():
        value, mag = want[key]
        column = key in ("dpost_weight", "dpre_weight") or (key == "dgate" and kind == "channel")
        kind_of = "f32" if column or (key == "dgate" and kind == "token") else dtype
        within(o, value, (256 + (T + 64 if column else 0)) * U * mag, kind_of)
        if o.dim() == 2:
            assert unmarked(o, 3.0)


@pytest.mark.parametrize("case", NORMS, ids=lambda c: "-".join(map(str, c)))
def test_norm_gradient(dfm, case):
    check_norm_grad(dfm, *case)


@pytest.mark.parametrize("case", [NORMS[2], NORMS[4], NORMS[7], NORMS[11]], ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("pad", [3, 8])
def test_norm_gradient_strides(dfm, case, pad):
    check_norm_grad(dfm, *case, pad=pad)


@pytest.mark.parametrize("kw", [dict(weights=False), dict(dh_too=False), dict(dn_too=False), dict(wanted=("du",)),
                                dict(wanted=("dresidual",)), dict(wanted=("dpre_weight",)), dict(wanted=("dgate",)),
                                dict(wanted=("dpost_weight", "dgate"))], ids=str)
@pytest.mark.parametrize("kind", ["channel", "token", "full"])
def test_norm_gradient_of_some(dfm, kind, kw):
    check_norm_grad(dfm, 333, 264, "bf16", "f32", True, kind, 1.0, **kw)


@pytest.mark.parametrize("case", [
    (170, 7168, "bf16", "f32", True, "channel", 1.0), (700, 2048, "f16", "f32", True, "full", 0.5), (1300, 1024, "bf16", "bf16", True, "token", 1.0),
    (1500, 520, "bf16", "f32", False, "channel", 1.0), (1250, 520, "f32", "f32", True, "full", -1.0), (620, 768, "f32", "f32", True, "channel", 1.0),
    (1217, 648, "f16", "f16", False, "none", 1.0),
], ids=lambda c: "-".join(map(str, c)))
def test_norms_through_the_ring(dfm, case):
    """Rows of every length that it takes, a few more than start at once."""
    check_norm(dfm, *case)
    check_norm_grad(dfm, *case)


def test_norm_gradient_in_place_and_without_rows(dfm):
    T, H, g = 50, 128, gen(0)
    dh, dn, u, h = (rows(T, H, g, "bf16") for _ in range(4))
    du, dr = torch.empty_like(u), torch.empty_like(u)
    dfm.block_norm_grad(dh, dn, u, h, "bf16", T, H, du, dr, post=True)
    dfm.block_norm_grad(dh, dn, u, h, "bf16", T, H, dn, dh, post=True)
    assert torch.equal(dn, du) and torch.equal(dh, dr)
    sums = torch.full((3, H), 3.0, device="cuda")
    dfm.block_norm_grad(None, None, None, None, "bf16", 0, H, post=True, dpost_weight=sums[0], dpre_weight=sums[1], gate=sums[2],
                        gate_kind="channel", dgate=sums[2], weight_dtype="f32")
    assert bool((sums == 0).all())


def test_norm_gradient_against_differences(dfm):
    T, H, g = 6, 40, gen(4)
    u, r, dh, dn = (rows(T, H, g, "f32") for _ in range(4))
    q, v, gate = (randn(H, g=g) for _ in range(3))
    h = torch.empty(T, H, device="cuda")
    dfm.block_norm(u, r, "f32", T, H, h, post=True, post_weight=q, gate=gate, gate_kind="channel", residual_scale=0.5, eps=EPS)
    grads = [torch.empty(T, H, device="cuda"), torch.empty(T, H, device="cuda")] + [torch.empty(H, device="cuda") for _ in range(3)]
    size = dfm.block_norm_grad_workspace(T, H)
    dfm.block_norm_grad(dh, dn, u, h, "f32", T, H, grads[0], grads[1], post=True, post_weight=q, dpost_weight=grads[2], gate=gate,
                        gate_kind="channel", dgate=grads[3], residual_scale=0.5, pre_weight=v, dpre_weight=grads[4], eps=EPS,
                        workspace=torch.empty(size, dtype=torch.uint8, device="cuda"), workspace_bytes=size)

    def loss(u, r, q, gate, v):
        _, h, n = forward64(u, r, True, q, gate, "channel", 0.5, v)
        return (h * dh.double() + n * dn.double()).sum().item()
    at = [t.double() for t in (u, r, q, gate, v)]
    for i, grad in enumerate(grads):
        d = torch.randn(grad.shape, generator=g, device="cuda", dtype=torch.float64)
        slope = (loss(*[t + 1e-5 * d if j == i else t for j, t in enumerate(at)])
                 - loss(*[t - 1e-5 * d if j == i else t for j, t in enumerate(at)])) / 2e-5
        # fp32 gradients: some 1e-6 of each; the difference's own error is of the order of its step squared
        assert abs((grad.double() * d).sum().item() - slope) <= 1e-5 * (grad.double().abs() * d.abs()).sum().item() + 1e-7


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H, T", [(1, 3), (48, 5), (1001, 5), (7168, 400), (8192, 3), (8192, 400), (32768, 3), (32767, 3)])
def test_norm_of_rows_at_the_types_end(dfm, dtype, H, T):
    """Rows whose squares overflow at any scale but a small one, and with an eps that
    overflows beside them; both norms and their gradients."""
    g = gen(H)
    sign = torch.where(torch.rand(T, H, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    x = sign * torch.finfo(DT[dtype]).max
    x[1] *= torch.rand(H, generator=g, device="cuda")
    x[2] = sign[2] * 1.3e38
    x = x.to(DT[dtype])
    for eps in (EPS, 3e38):
        xd = x.double()
        h, n = torch.empty_like(x), torch.empty_like(x)
        if eps > 1:
            x[0] = x[0] * 2.0 ** -65  # squares of 8e37, finite without eps where H is small
            xd = x.double()
        rms = torch.rsqrt((xd * xd).mean(1, keepdim=True) + eps)
        dfm.block_norm(x, None, dtype, T, H, h, n, post=True, eps=eps)
        want = xd * rms
        # rms is below 2^-126 where x is largest, and loses three bits
        within(h, want, 64 * U * want.abs(), dtype)
        dfm.block_norm(None, x, dtype, T, H, n=n, eps=eps)
        within(n, want, 64 * U * want.abs(), dtype)
        # gradients a row, of both norms: dn large, so that the results are no subnormals
        dn = (1e30 * torch.randn(T, H, generator=g, device="cuda")).to(DT[dtype])
        dx, du = torch.empty_like(x), torch.empty_like(x)
        hat, dd = want, dn.double()
        grad = rms * (dd - hat * (dd * hat).mean(1, keepdim=True))
        bound = rms * (128 + math.ceil(H / 256)) * U * (dd.abs() + hat.abs() * (dd * hat).abs().mean(1, keepdim=True))
        dfm.block_norm_grad(None, dn, None, x, dtype, T, H, dresidual=dx, eps=eps)
        within(dx, grad, bound, dtype)
        dfm.block_norm_grad(dn, None, x, None, dtype, T, H, du=du, post=True, eps=eps)
        within(du, grad, bound, dtype)


@pytest.mark.parametrize("kind", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("H, T, dtype", [(64, 5, "f32"), (61, 5, "f32"), (64, 5, "bf16"), (2048, 400, "bf16"), (1024, 700, "f32"), (9000, 3, "bf16"),
                                         (16384, 2, "f32")])
def test_norm_gradient_whose_cross_sums_overflow(dfm, H, T, dtype, post, kind):
    """u q g h and u q g y add up beyond fp32 where neither the squares of u nor h do."""
    g = gen(H + T)

    def most(size):  # values of one size and either sign
        return (size * (0.5 + torch.rand(T, H, generator=g, device="cuda"))).to(DT[dtype])
    big = 2.0 ** 63.5 / H ** 0.5  # squares that add up to a quarter of fp32's range and so
    u, h = most(big / 1.5), most(big / 1.5)
    dn, dh = most(0.1), most(1e-18)
    u[-1], dn[-1], dh[-1] = u[-1] * 2.0 ** -30, dn[-1] * 1e28, dh[-1] * 1e3  # the sums with y alone
    q = torch.full((H,), 3.0, device="cuda") if post else None
    v = torch.full((H,), 2.0, device="cuda")
    gate = {"none": None, "channel": torch.full((H,), 2.0, device="cuda"), "token": torch.full((T,), 2.0, device="cuda"),
            "full": torch.full((T, H), 2.0, device="cuda").to(DT[dtype])}[kind]
    out = dict(du=torch.empty_like(u), dresidual=torch.empty_like(u), dpre_weight=torch.empty(H, device="cuda"))
    if post:
        out["dpost_weight"] = torch.empty(H, device="cuda")
    if kind != "none":
        out["dgate"] = torch.empty_like(gate)
    size = dfm.block_norm_grad_workspace(T, H)
    dfm.block_norm_grad(dh, dn, u, h, dtype, T, H, post=post, post_weight=q, gate=gate, gate_kind=kind, pre_weight=v, eps=EPS,
                        workspace=torch.empty(size, dtype=torch.uint8, device="cuda"), workspace_bytes=size, **out)
    want = grad64(dh.double(), dn.double(), u.double(), h.double(), post, q, gate, kind, 1.0, v)
    for key, o in out.items():
        value, mag = want[key]
        column = key in ("dpost_weight", "dpre_weight") or (key == "dgate" and kind == "channel")
        kind_of = "f32" if column or (key == "dgate" and kind == "token") else dtype
        assert bool((value.abs() < torch.finfo(DT[kind_of]).max).all()), key
        within(o, value, (256 + (T + 64 if column else 0)) * U * mag, kind_of)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("H, T, dtype", [(64, 6, "f32"), (61, 6, "f32"), (2048, 420, "bf16"), (1024, 700, "f32"), (9000, 6, "bf16")])
def test_norm_gradient_of_rows_far_apart_in_size(dfm, H, T, dtype, post):
    """h beyond fp32's root next to a small u, and the other way about: either is summed
    at a scale of its own."""
    g = gen(H)
    size = torch.tensor([[1e-20, 1e30], [1e30, 1e-20], [1.0, 3e38], [3e38, 1.0], [1e-30, 1e19], [3e19, 3e19]], device="cuda")
    size = size.repeat(-(-T // 6), 1)[:T]
    lot = [(torch.randn(T, H, generator=g, device="cuda").clamp(-1, 1) * s).to(DT[dtype])
           for s in (size[:, :1], size[:, 1:], torch.ones(T, 1, device="cuda"), 1e-15 * torch.ones(T, 1, device="cuda"))]
    u, h, dn, dh = lot
    q, gate = torch.full((H,), 1.5, device="cuda") if post else None, torch.full((T,), 0.5, device="cuda")
    out = dict(du=torch.empty_like(u), dresidual=torch.empty_like(u), dgate=torch.empty(T, device="cuda"))
    dfm.block_norm_grad(dh, dn, u, h, dtype, T, H, post=post, post_weight=q, gate=gate, gate_kind="token", eps=EPS, **out)
    want = grad64(dh.double(), dn.double(), u.double(), h.double(), post, q, gate, "token", 1.0, None)
    for key, o in out.items():
        value, mag = want[key]
        # not the gate's gradient of 61 terms of 3e38 times some 0.3 and more (6e39 of magnitudes, which no fp32 sum holds)
        there = mag < torch.finfo(torch.float32).max
        within(o[there], value[there], 256 * U * mag[there], "f32" if key == "dgate" else dtype)


# ---- balance ----------------------------------------------------------------
def balance64(z, ids, k, E, offs, mask, score, coef, z_coef, dloss=None, weights=None, dweights=None):
    T, S = z.shape[0], len(offs) - 1
    loss, counts, tokens, probs = [], [], [], []
    d, touched = torch.zeros_like(z), torch.zeros(T, dtype=torch.bool, device=z.device)
    for s in range(S):
        at = torch.arange(offs[s], max(offs[s], offs[s + 1]), device=z.device)
        touched[at] = True
        at = at[mask[at]]
        n = at.numel()
        tokens.append(n)
        if n == 0:
            loss.append(0.0)
            counts.append(torch.zeros(E, dtype=torch.int64, device=z.device))
            probs.append(torch.zeros(E, dtype=torch.float64, device=z.device))
            continue
        x, i = z[at], ids[at].long()
        closed = torch.isneginf(x).all(1, keepdim=True)
        a = torch.nn.functional.logsigmoid(x) if score == "sigmoid" else x
        p = torch.where(closed, 0.0, torch.softmax(a, 1))
        soft = torch.where(closed, 0.0, torch.softmax(x, 1))
        l = torch.where(closed[:, 0], 0.0, torch.logsumexp(x, 1))
        m = torch.sigmoid(-x) if score == "sigmoid" else torch.ones_like(x)
        there = (i >= 0) & (i < E)
        c = torch.bincount(i[there], minlength=E)
        f = c.double() * E / (k * n)
        counts.append(c)
        probs.append(p.mean(0))
        loss.append(coef * (f @ probs[-1]).item() + z_coef * l.square().mean().item())
        if dloss is not None:
            g = dloss[s].double() * (coef / n * p * m * (f - (p @ f)[:, None]) + 2 * z_coef / n * l[:, None] * soft)
            if weights is not None:
                w, dw = weights[at].double() * there, dweights[at].double()
                kept = w * (dw - (w * dw).sum(1, keepdim=True))
                g = g + m * torch.zeros_like(x).scatter_add_(1, i.clamp(0, E - 1), kept)
            d[at] = g
    return torch.tensor(loss, dtype=torch.float64, device=z.device), torch.stack(counts), tokens, torch.stack(probs), d, touched


BALANCE = [
    # T, E, k, dtype, score, S, mask
    (1, 1, 1, "f32", "softmax", 1, 0.0), (1, 896, 16, "f32", "softmax", 1, 0.0), (8, 8, 2, "bf16", "sigmoid", 1, 0.0),
    (64, 896, 16, "f32", "sigmoid", 3, 0.2), (33, 61, 6, "f16", "softmax", 5, 0.5), (300, 128, 8, "f32", "softmax", 1, 0.0),
    (301, 129, 7, "f32", "sigmoid", 300, 0.1), (1000, 255, 32, "bf16", "softmax", 7, 0.0), (5000, 1024, 4, "f32", "softmax", 2, 0.0),
    (4097, 512, 9, "f16", "sigmoid", 11, 0.9), (9000, 33, 3, "f32", "softmax", 1000, 0.0), (20000, 64, 8, "bf16", "sigmoid", 1, 0.0),
    (7000, 897, 16, "f32", "softmax", 4, 0.0),
]


def check_balance(dfm, T, E, k, dtype, score, S, drop, pad=0, closed=False):
    g = gen(T + E)
    z = rows(T, E, g, dtype, pad, sigma=2.0)
    mask = (torch.rand(T, generator=g, device="cuda") >= drop)
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < 0.1, torch.tensor(-1, device="cuda", dtype=torch.int32), ids)
    if T > 2:
        ids[0, 0], ids[1, -1] = E, -2 ** 31
    if closed:
        z[torch.rand(T, E, generator=g, device="cuda") < 0.3] = float("-inf")
        z[::5] = float("-inf")
    zd = z.double()
    if drop:
        z[~mask] = float("nan")
    lead, tail = (T // 7, T // 9) if S > 1 else (0, 0)
    cut = torch.randint(lead, T - tail + 1, (S - 1,), generator=g, device="cuda").sort().values.tolist() if S > 1 else []
    at = [lead] + cut + [T - tail]
    offs = torch.tensor(at, dtype=torch.int32, device="cuda") if S > 1 else None
    m8 = mask.to(torch.uint8) if drop else None
    loss, probs = torch.full((S,), 3.0, device="cuda"), torch.full((S, E), 3.0, device="cuda")
    counts, tokens = torch.full((S, E), 7, dtype=torch.int32, device="cuda"), torch.full((S,), 7, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    size = dfm.balance_loss_workspace(T, E, S)
    workspace = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    coef, z_coef = 0.5, 0.01
    kw = dict(offs=offs, S=S, mask=m8, score=score, coef=coef, z_coef=z_coef, ldl=z.stride(0))
    dfm.balance_loss(z, dtype, T, E, ids, k, loss, counts, tokens, workspace, size, probs=probs, status=status, **kw)
    dloss = randn(S, g=g)
    w = torch.rand(T, k, generator=g, device="cuda")
    w, dw = w / w.sum(1, keepdim=True), randn(T, k, g=g, sigma=0.01)
    dz = rows(T, E, g, dtype, pad, mark=3.0)
    dfm.balance_loss_grad(dloss, z, dtype, T, E, ids, k, counts, tokens, dz, weights=w, dweights=dw, lddl=dz.stride(0), **kw)
    want = balance64(zd, ids, k, E, at, mask, score, coef, z_coef, dloss, w, dw)
    assert status.item() == 0
    assert torch.equal(counts.long(), want[1]) and tokens.tolist() == want[2]
    # a probability: its exponent's argument is off by 3 U of |z| <= 16 or so, expf, the sum (42 additions) and the quotient
    rel = 128 * U
    n = torch.tensor(want[2], device="cuda").clamp(min=1)[:, None]
    within(probs, want[3], (rel + (T / 1000 + 512) * U) * want[3], "f32")
    f = want[1].double() * E / (k * n)
    size64 = coef * (f * want[3]).sum(1) + z_coef * 300  # logsumexp is below 17
    within(loss, want[0], (rel + (T / 1000 + 600) * U) * size64, "f32")
    # the gradient: terms of p (|f| + f p) coef / n, l p, and the routing weights', each off by rel and what f p is off
    most = balance64(zd, ids, k, E, at, mask, score, coef, z_coef, dloss.abs(), w, dw.abs())[4].abs()
    seq = torch.searchsorted(torch.tensor(at[1:], device="cuda"), torch.arange(T, device="cuda"), right=True).clamp(max=S - 1)
    p = torch.nan_to_num(torch.softmax(torch.nn.functional.logsigmoid(zd) if score == "sigmoid" else zd, 1))
    fp = (f[seq] * p).sum(1, keepdim=True)
    each = dloss.abs().double()[seq][:, None] / n[seq]
    kept = torch.zeros_like(zd).scatter_add_(1, ids.long().clamp(0, E - 1), (w * (dw.abs() + (w * dw.abs()).sum(1, keepdim=True))).double())
    soft = torch.nan_to_num(torch.softmax(zd, 1))
    mag = each * (coef * p * (f[seq] + fp) + 2 * z_coef * 17 * soft) + kept + most
    assert bool((dz[~want[5]] == 3).all())
    inside = want[5]
    within(dz[inside], want[4][inside], 4 * rel * mag[inside], dtype)
    assert bool((dz[inside & ~mask] == 0).all()) and unmarked(dz, 3.0)


@pytest.mark.parametrize("case", BALANCE, ids=lambda c: "-".join(map(str, c)))
def test_balance(dfm, case):
    check_balance(dfm, *case)


@pytest.mark.parametrize("case", [BALANCE[3], BALANCE[4], BALANCE[6], BALANCE[7]], ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("pad", [1, 4])
def test_balance_strides(dfm, case, pad):
    check_balance(dfm, *case, pad=pad)


@pytest.mark.parametrize("case", [BALANCE[3], BALANCE[4], BALANCE[5]], ids=lambda c: "-".join(map(str, c)))
def test_balance_with_experts_that_are_not_allowed(dfm, case):
    check_balance(dfm, *case, closed=True)


@pytest.mark.parametrize("T, E, k, dtype, drop", [
    (2, 896, 32, "f32", 0.0), (17, 300, 5, "bf16", 0.3), (64, 1024, 8, "f32", 0.1), (127, 897, 16, "f16", 0.0), (128, 896, 16, "f32", 0.5),
    (129, 896, 16, "f32", 0.1), (100, 128, 9, "bf16", 0.0), (129, 128, 9, "f32", 0.0), (200, 64, 32, "f32", 0.2), (257, 61, 12, "f16", 0.1),
    (512, 32, 32, "f32", 0.1), (513, 20, 20, "bf16", 0.0), (40, 3, 32, "f32", 0.1), (40, 1, 32, "f32", 0.0), (5, 1024, 3, "f32", 1.0),
])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_of_few_rows(dfm, T, E, k, dtype, drop, score):
    """Rows of one sequence that a cluster finishes, and just above; tokens that
    name an expert many times, over several lots of a row's lanes."""
    check_balance(dfm, T, E, k, dtype, score, 1, drop)


@pytest.mark.parametrize("T, E", [(60, 20), (700, 100), (700, 900)])
def test_balance_gradient_in_place(dfm, T, E):
    g = gen(T + E)
    z, ids = randn(T, E, g=g), torch.randint(0, E, (T, 4), generator=g, device="cuda", dtype=torch.int32)
    loss, counts, tokens = torch.empty(1, device="cuda"), torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    size = dfm.balance_loss_workspace(T, E, 1)
    kw = dict(coef=0.5, z_coef=0.01)
    dfm.balance_loss(z, "f32", T, E, ids, 4, loss, counts, tokens, torch.empty(size, dtype=torch.uint8, device="cuda"), size, **kw)
    one, want = torch.ones(1, device="cuda"), torch.empty_like(z)
    dfm.balance_loss_grad(one, z, "f32", T, E, ids, 4, counts, tokens, want, **kw)
    dfm.balance_loss_grad(one, z, "f32", T, E, ids, 4, counts, tokens, z, **kw)
    assert torch.equal(z, want)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shift", [-1e4, -200.0, 200.0, 1e4])
def test_balance_of_far_logits(dfm, score, shift):
    """Scores that are all tiny, or all one, keep their ratios."""
    T, E, k = 40, 24, 2
    g = gen(2)
    z = randn(T, E, g=g) + shift
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    loss, probs = torch.empty(1, device="cuda"), torch.empty(1, E, device="cuda")
    counts, tokens = torch.empty(1, E, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    size = dfm.balance_loss_workspace(T, E)
    dfm.balance_loss(z, "f32", T, E, ids, k, loss, counts, tokens, torch.empty(size, dtype=torch.uint8, device="cuda"), size, probs=probs,
                     score=score)
    want = balance64(z.double(), ids, k, E, [0, T], torch.ones(T, dtype=torch.bool, device="cuda"), score, 1.0, 0.0)
    within(probs, want[3], 256 * U * want[3], "f32")
    within(loss, want[0], 512 * U * want[0], "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("E", [16, 300])
def test_balance_of_scores_that_are_nothing_beside_the_largest(dfm, dtype, E):
    """A sigmoid's score below 2^-126 of the largest is 0, and its logit's
    gradient is the routing weight's alone."""
    z = torch.full((1, E), -200.0, device="cuda")
    z[0, :9] = torch.tensor([0.0, -50.0, -86.0, -89.0, -104.0, -1e3, -6e4, float("-inf"), 1.0])
    z = z.to(DT[dtype])
    ids = torch.tensor([[0, 1, 4, 7, 8]], dtype=torch.int32, device="cuda")
    k = ids.shape[1]
    loss, probs = torch.empty(1, device="cuda"), torch.empty(1, E, device="cuda")
    counts, tokens = torch.empty(1, E, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    size = dfm.balance_loss_workspace(1, E)
    dfm.balance_loss(z, dtype, 1, E, ids, k, loss, counts, tokens, torch.empty(size, dtype=torch.uint8, device="cuda"), size, probs=probs,
                     score="sigmoid")
    w, dw = torch.full((1, k), 1 / k, device="cuda"), torch.tensor([[1.0, -2.0, 3.0, 5.0, 7.0]], device="cuda")
    dz = torch.empty_like(z)
    dfm.balance_loss_grad(torch.ones(1, device="cuda"), z, dtype, 1, E, ids, k, counts, tokens, dz, weights=w, dweights=dw, score="sigmoid")
    every = torch.ones(1, dtype=torch.bool, device="cuda")
    want = balance64(z.double(), ids, k, E, [0, 1], every, "sigmoid", 1.0, 0.0, torch.ones(1, device="cuda"), w, dw)
    # (an exponent of size 104 is rounded: 104 U)
    assert bool(((probs.double() - want[3]).abs() <= 256 * U * want[3] + 2.0 ** -125).all())
    within(dz, want[4], 512 * U * (want[4].abs() + want[3] * E) + 2.0 ** -120, dtype)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("E", [6, 24, 61, 200, 896])
def test_balance_of_logits_at_the_types_ends(dfm, score, dtype, E):
    """The type's lowest value stands for an expert that is not allowed, the lowest
    in the whole row for a token that no expert may have: uniform, by the
    definition. Each row a sequence, then all of them one."""
    g = gen(E)
    low, high = torch.finfo(DT[dtype]).min, torch.finfo(DT[dtype]).max
    z = randn(16, E, g=g)
    z[0], z[1] = low, high
    z[2, 1:] = low
    z[3], z[3, E // 2] = low, high
    z[4], z[4, 0] = float("-inf"), low
    z[5], z[5, 1] = low, float("-inf")
    z[6], z[7] = 0.7 * low, 0.7 * high  # about where a product with log2(e) leaves fp32
    z[8], z[9] = 0.6 * low, 0.6 * high
    z[10, ::2] = low
    z[11] = low
    z[11, -1] = 0.9 * low
    z[12, ::3] = high
    z[13], z[13, E - 1] = 0.9 * high, 0.8 * high
    z[14, E // 3] = low
    z = z.to(DT[dtype])
    zd, T, k = z.double(), z.shape[0], 3
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    for S, at in ((T, list(range(T + 1))), (1, [0, T])):
        offs = torch.tensor(at, dtype=torch.int32, device="cuda") if S > 1 else None
        loss, probs = torch.empty(S, device="cuda"), torch.empty(S, E, device="cuda")
        counts, tokens = torch.empty(S, E, dtype=torch.int32, device="cuda"), torch.empty(S, dtype=torch.int32, device="cuda")
        size = dfm.balance_loss_workspace(T, E, S)
        kw = dict(offs=offs, S=S, score=score, coef=0.5)
        dfm.balance_loss(z, dtype, T, E, ids, k, loss, counts, tokens, torch.empty(size, dtype=torch.uint8, device="cuda"), size,
                         probs=probs, **kw)
        every = torch.ones(T, dtype=torch.bool, device="cuda")
        want = balance64(zd, ids, k, E, at, every, score, 0.5, 0.0)
        within(probs, want[3], 256 * U * want[3], dtype="f32")
        f = want[1].double() * E / (k * torch.tensor(want[2], device="cuda")[:, None])
        within(loss, want[0], 512 * U * 0.5 * (f * want[3]).sum(1), "f32")
        # the gradient, without and with the squared logsumexp's part: terms of p (f + f p), l p and the routing weights'
        dloss, w, dw = torch.ones(S, device="cuda"), torch.full((T, k), 1 / k, device="cuda"), randn(T, k, g=g)
        for z_coef in (0.0, 1e-3):
            dz = torch.empty_like(z)
            dfm.balance_loss_grad(dloss, z, dtype, T, E, ids, k, counts, tokens, dz, weights=w, dweights=dw, z_coef=z_coef, **kw)
            grad = balance64(zd, ids, k, E, at, every, score, 0.5, z_coef, dloss, w, dw)[4]
            p = torch.softmax(torch.nn.functional.logsigmoid(zd) if score == "sigmoid" else zd, 1)
            seq = torch.arange(T, device="cuda") if S > 1 else torch.zeros(T, dtype=torch.int64, device="cuda")
            n = torch.tensor(want[2], device="cuda").double()[seq][:, None]
            mag = 0.5 / n * p * (f[seq] + (f[seq] * p).sum(1, keepdim=True))
            mag = mag + 2 * z_coef / n * torch.logsumexp(zd, 1, keepdim=True).abs() * torch.softmax(zd, 1)
            kept = (w * (dw.abs() + (w * dw.abs()).sum(1, keepdim=True))).double()
            mag = mag + torch.zeros_like(zd).scatter_add_(1, ids.long(), kept)
            within(dz, grad, 512 * U * mag, dtype)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("far", [3e6, 1e8, 1e9, 1e10, 1e13, 1e30])
def test_balance_of_logits_whose_spacing_is_wide(dfm, score, far):
    """Rows about as far as their values lie apart: where an exponent's rounding is
    more than the exponent."""
    T, E, k = 40, 24, 2
    g = gen(3)
    step = max(1.0, 2.0 ** math.floor(math.log2(far) - 23))
    z = torch.randint(-20, 3, (T, E), generator=g, device="cuda").double() * step
    z = (z + torch.where(torch.arange(T, device="cuda") % 2 == 0, far, -far)[:, None]).float()
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    offs = torch.arange(T + 1, dtype=torch.int32, device="cuda")
    loss, probs = torch.empty(T, device="cuda"), torch.empty(T, E, device="cuda")
    counts, tokens = torch.empty(T, E, dtype=torch.int32, device="cuda"), torch.empty(T, dtype=torch.int32, device="cuda")
    size = dfm.balance_loss_workspace(T, E, T)
    kw = dict(offs=offs, S=T, score=score)
    dfm.balance_loss(z, "f32", T, E, ids, k, loss, counts, tokens, torch.empty(size, dtype=torch.uint8, device="cuda"), size, probs=probs,
                     z_coef=1e-60 ** 0.5, **kw)
    every, one = torch.ones(T, dtype=torch.bool, device="cuda"), torch.ones(T, device="cuda")
    want = balance64(z.double(), ids, k, E, list(range(T + 1)), every, score, 1.0, 1e-60 ** 0.5, one)
    within(probs, want[3], 256 * U * want[3], "f32")
    if far < 1e18:  # where the square of the logarithm stays in fp32
        within(loss, want[0], 512 * U * want[0], "f32")
    dz = torch.empty_like(z)
    dfm.balance_loss_grad(one, z, "f32", T, E, None, k, counts, tokens, dz, z_coef=1e-60 ** 0.5, **kw)
    f = want[1].double() * E / k
    # an exponential below 2^-126 is 0: as much of each f is missing (e^-88 = 6.1e-39 times f = 12 is 7.3e-38)
    terms = f + (f * want[3]).sum(1, keepdim=True)
    mag = want[3] * terms + 2e-30 * far * torch.softmax(z.double(), 1)
    within(dz, want[4], 512 * U * mag + 2.0 ** -126 * terms, "f32")


def test_balance_counts_more_tokens_than_fp32_does(dfm):
    T, E = 2 ** 24 + 3, 2
    z = torch.zeros(T, E, device="cuda")
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    ids[5] = 1
    loss, probs = torch.empty(1, device="cuda"), torch.empty(1, E, device="cuda")
    counts, tokens = torch.empty(1, E, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    size = dfm.balance_loss_workspace(T, E)
    dfm.balance_loss(z, "f32", T, E, ids, 1, loss, counts, tokens, torch.empty(size, dtype=torch.uint8, device="cuda"), size, probs=probs)
    assert tokens.item() == T and counts.tolist() == [[T - 1, 1]]
    # halves: every partial sum is exact in fp32 but the last few
    assert bool(((probs.double() - 0.5).abs() <= 64 * U).all()) and abs(loss.item() - 1.0) <= 128 * U


@pytest.mark.parametrize("S", [1, 2, 31, 32, 33, 1023, 1025, 40000])
def test_balance_finds_every_sequence(dfm, S):
    """One token each, then two in the last: sequence s has expert s % E alone."""
    E, T = 8, S + 1
    of = torch.arange(T, device="cuda").clamp(max=S - 1)
    ids = (of % E).to(torch.int32)[:, None].contiguous()
    offs = torch.cat([torch.arange(S, device="cuda"), torch.tensor([T], device="cuda")]).to(torch.int32)
    z = torch.zeros(T, E, device="cuda")
    loss = torch.empty(S, device="cuda")
    counts, tokens = torch.empty(S, E, dtype=torch.int32, device="cuda"), torch.empty(S, dtype=torch.int32, device="cuda")
    size = dfm.balance_loss_workspace(T, E, S)
    dfm.balance_loss(z, "f32", T, E, ids, 1, loss, counts, tokens, torch.empty(size, dtype=torch.uint8, device="cuda"), size, offs=offs, S=S)
    want = torch.zeros(S, E, dtype=torch.int32, device="cuda").index_put_((of, of % E), torch.ones(T, dtype=torch.int32, device="cuda"),
                                                                         accumulate=True)
    assert torch.equal(counts, want) and torch.equal(tokens.long(), want.sum(1))
    d = torch.empty_like(z)
    dfm.balance_loss_grad(torch.ones(S, device="cuda"), z, "f32", T, E, None, 1, counts, tokens, d, offs=offs, S=S)
    n = want.sum(1)[of][:, None].double()
    f = torch.zeros(T, E, dtype=torch.float64, device="cuda").scatter_(1, (of % E)[:, None], float(E))
    within(d, (f - 1) / E / n, 64 * U * (f + 1) / E / n, "f32")


def test_balance_all_masked_and_no_rows(dfm):
    T, E, k, S = 30, 40, 2, 3
    for rows_there in (T, 0):
        z = torch.full((T, E), float("nan"), device="cuda")
        mask = torch.zeros(T, dtype=torch.uint8, device="cuda")
        offs = torch.tensor([0, 10, 10, rows_there and 25], dtype=torch.int32, device="cuda").clamp(max=rows_there)
        loss, probs = torch.full((S,), 3.0, device="cuda"), torch.full((S, E), 3.0, device="cuda")
        counts, tokens = torch.full((S, E), 7, dtype=torch.int32, device="cuda"), torch.full((S,), 7, dtype=torch.int32, device="cuda")
        size = dfm.balance_loss_workspace(T, E, S)
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        dfm.balance_loss(z, "f32", rows_there, E, torch.zeros(T, k, dtype=torch.int32, device="cuda"), k, loss, counts, tokens, ws, size,
                         probs=probs, offs=offs, S=S, mask=mask)
        assert not bool(loss.any() | probs.any() | counts.any() | tokens.any())
        dz = torch.full((T, E), 3.0, device="cuda")
        dfm.balance_loss_grad(loss, z, "f32", rows_there, E, None, k, counts, tokens, dz, offs=offs, S=S, mask=mask)
        assert bool((dz[:25 if rows_there else 0] == 0).all()) and bool((dz[25 if rows_there else 0:] == 3).all())


@pytest.mark.parametrize("at", [[0, 30, 20, 50], [-5, 10, 20, 50], [0, 10, 20, 99], [60, 50, 10, 0]])
def test_balance_reports_sequences_out_of_order(dfm, at):
    T, E, k, S = 50, 20, 2, 3
    g = gen(1)
    z, ids = randn(T, E, g=g), torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    offs = torch.tensor(at, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss = torch.zeros(S, device="cuda")
    counts, tokens = torch.zeros(S, E, dtype=torch.int32, device="cuda"), torch.zeros(S, dtype=torch.int32, device="cuda")
    size = dfm.balance_loss_workspace(T, E, S)
    ws = torch.zeros(size + 64, dtype=torch.uint8, device="cuda")
    dfm.balance_loss(z, "f32", T, E, ids, k, loss, counts, tokens, ws, size, offs=offs, S=S, status=status)
    assert status.item() == 1 and not bool(ws[size:].any())
    out = torch.full((T + 2, E), 3.0, device="cuda")
    dfm.balance_loss_grad(loss, z, "f32", T, E, None, k, counts, tokens, out[1:-1], offs=offs, S=S)
    assert bool((out[0] == 3).all()) and bool((out[-1] == 3).all())


def test_balance_gradient_against_differences(dfm):
    T, E, k = 12, 10, 3
    for score in ("softmax", "sigmoid"):
        g = gen(6)
        z = randn(T, E, g=g)
        top = z.topk(k, 1)
        ids = top.indices.to(torch.int32).contiguous()
        coef, z_coef, dw = 0.7, 0.1, randn(T, k, g=g)

        def routing(z):
            kept = (torch.sigmoid(z) if score == "sigmoid" else torch.exp(z)).gather(1, ids.long())
            return kept / kept.sum(1, keepdim=True)
        w = routing(z.double()).float()
        loss, dz = torch.empty(1, device="cuda"), torch.empty(T, E, device="cuda")
        counts, tokens = torch.empty(1, E, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
        size = dfm.balance_loss_workspace(T, E)
        kw = dict(score=score, coef=coef, z_coef=z_coef)
        dfm.balance_loss(z, "f32", T, E, ids, k, loss, counts, tokens, torch.empty(size, dtype=torch.uint8, device="cuda"), size, **kw)
        dloss = torch.tensor([1.5], device="cuda")
        dfm.balance_loss_grad(dloss, z, "f32", T, E, ids, k, counts, tokens, dz, weights=w, dweights=dw, **kw)
        every = torch.ones(T, dtype=torch.bool, device="cuda")

        def value(z):
            return 1.5 * balance64(z, ids, k, E, [0, T], every, score, coef, z_coef)[0].item() + (routing(z) * dw.double()).sum().item()
        d = torch.randn(T, E, generator=g, device="cuda", dtype=torch.float64)
        slope = (value(z.double() + 1e-5 * d) - value(z.double() - 1e-5 * d)) / 2e-5
        assert abs((dz.double() * d).sum().item() - slope) <= 1e-5 * (dz.double().abs() * d.abs()).sum().item() + 1e-7


# ---- together ---------------------------------------------------------------
class Block:
    """One block around frozen routed experts: norm, router product, balance
    loss, tokens to their experts and back, a gated shared expert, and the norm
    behind it all; and its backward, through the library alone."""

    T, H, I, E, k = 96, 256, 128, 16, 4

    def __init__(self, dfm, seed):
        T, H, I, E, k = self.T, self.H, self.I, self.E, self.k
        g, bf = gen(seed), "bf16"
        self.dfm, dev = dfm, "cuda"
        self.x = rows(T, H, g, bf)
        self.v, self.q = 1 + randn(H, g=g, sigma=0.1), 1 + randn(H, g=g, sigma=0.1)
        self.router = randn(E, H, g=g, dtype=bf, sigma=H ** -0.5)
        self.w1, self.w2 = randn(2 * I, H, g=g, dtype=bf, sigma=H ** -0.5), randn(H, I, g=g, dtype=bf, sigma=I ** -0.5)
        self.dn = randn(T, H, g=g, dtype=bf, sigma=0.1)
        e = lambda *s, t=torch.bfloat16: torch.empty(*s, dtype=t, device=dev)  # noqa: E731
        f = torch.float32
        self.n, self.logits, self.z, self.a, self.u = e(T, H), e(T, E, t=f), e(T, 2 * I), e(T, I), e(T, H)
        self.h, self.out = e(T, H), e(T, H)
        self.ids, self.w = e(T, k, t=torch.int32), e(T, k, t=f)
        self.loss, self.counts, self.tokens = e(1, t=f), e(1, E, t=torch.int32), e(1, t=torch.int32)
        self.rows, self.offs, self.pos, self.src = e(T * k, H), e(E + 1, t=torch.int32), e(T * k, t=torch.int32), e(T * k, t=torch.int32)
        self.bal = e(dfm.balance_loss_workspace(T, E), t=torch.uint8)
        self.ws = e(dfm.block_norm_grad_workspace(T, H), t=torch.uint8)
        self.dh, self.du, self.dq, self.dv = e(T, H), e(T, H), e(H, t=f), e(H, t=f)
        self.dloss = torch.ones(1, device=dev)
        self.da, self.dz, self.dw2, self.dw1, self.dns = e(T, I), e(T, 2 * I), e(H, I, t=f), e(2 * I, H, t=f), e(T, H)
        self.drows, self.dwts, self.dlogits, self.dnr = e(T * k, H), e(T, k, t=f), e(T, E), e(T, H)
        self.drouter, self.dne, self.l16 = e(E, H, t=f), e(T, H), e(T, E)

    def forward(self):
        d, T, H, I, E, k = self.dfm, self.T, self.H, self.I, self.E, self.k
        d.block_norm(None, self.x, "bf16", T, H, n=self.n, pre_weight=self.v)
        d.matmul(self.n, self.router, "bf16", T, E, H, self.l16, "bf16")
        self.logits.copy_(self.l16)
        top = self.logits.topk(k, 1)
        self.ids.copy_(top.indices)
        self.w.copy_(torch.softmax(top.values, 1))
        d.balance_loss(self.l16, "bf16", T, E, self.ids, k, self.loss, self.counts, self.tokens, self.bal, self.bal.numel(), coef=0.1)
        d.permute(self.ids, T, k, E, self.n, "bf16", H, self.rows, self.offs, self.pos, self.src)
        d.unpermute(self.rows, "bf16", T * k, self.pos, self.w, T, k, H, self.u)  # experts that hand their rows on
        d.matmul(self.n, self.w1, "bf16", T, I, H, self.a, "bf16", act="swiglu", pre=self.z)
        d.matmul(self.a, self.w2, "bf16", T, H, I, self.u, "bf16", residual=self.u)
        d.block_norm(self.u, self.x, "bf16", T, H, self.h, self.out, post=True, post_weight=self.q)

    def backward(self):
        d, T, H, I, E, k = self.dfm, self.T, self.H, self.I, self.E, self.k
        d.block_norm_grad(None, self.dn, self.u, self.h, "bf16", T, H, self.du, self.dh, post=True, post_weight=self.q,
                          dpost_weight=self.dq, workspace=self.ws, workspace_bytes=self.ws.numel())
        d.matmul_grad(self.du, self.a, self.w2, "bf16", T, H, I, dx=self.da, dw=self.dw2)
        d.matmul_grad(self.da, self.n, self.w1, "bf16", T, I, H, dx=self.dns, dw=self.dw1, act="swiglu", pre=self.z, dz=self.dz)
        d.unpermute_grad(self.du, self.rows, "bf16", T * k, self.pos, self.w, T, k, H, self.drows, self.dwts)
        d.permute_grad(self.drows, "bf16", T * k, self.pos, T, k, H, self.dne)
        d.balance_loss_grad(self.dloss, self.l16, "bf16", T, E, self.ids, k, self.counts, self.tokens, self.dlogits, coef=0.1,
                            weights=self.w, dweights=self.dwts)
        d.matmul_grad(self.dlogits, self.n, self.router, "bf16", T, E, H, dx=self.dnr, dw=self.drouter)

    def loss64(self, x, router, w1, w2, v, q):
        """What the backward differentiates, in 64 bits (the chosen experts fixed)."""
        T, I, E, k = self.T, self.I, self.E, self.k
        n = x * rms64(x) * v
        z = n @ router.t()
        w = torch.softmax(z.gather(1, self.ids.long()), 1)
        f = self.counts[0].double() * E / (k * T)
        balance = 0.1 * (f @ torch.softmax(z, 1).mean(0))
        u = n * w.sum(1, keepdim=True) + act64(n @ w1.t(), "swiglu", I) @ w2.t()
        h = x + u * rms64(u) * q
        return balance + (h * rms64(h) * self.dn.double()).sum()

    def grads(self):
        return {"router": self.drouter, "w1": self.dw1, "w2": self.dw2, "q": self.dq}


def test_a_blocks_training_step(dfm):
    """Every weight's gradient against the 64-bit definition's, by autograd of
    torch: relative to its norm, for bf16 values between the calls (each
    rounding 2^-9, some eight of them in a row)."""
    b = Block(dfm, 11)
    b.forward()
    b.backward()
    leaves = {"x": b.x, "router": b.router, "w1": b.w1, "w2": b.w2, "v": b.v, "q": b.q}
    leaves = {key: t.double().requires_grad_() for key, t in leaves.items()}
    b.loss64(**leaves).backward()
    for key, got in b.grads().items():
        want = leaves[key].grad
        assert ((got.double() - want).norm() / want.norm()).item() <= 8 * 2.0 ** -9, key


def test_a_blocks_step_replays_from_a_graph(dfm):
    """Captured on a stream, replayed with other inputs: the eager bits. An eager
    copy of the block lives on meanwhile."""
    eager, b, other = Block(dfm, 1), Block(dfm, 1), Block(dfm, 2)
    other.forward()
    eager.forward()
    eager.backward()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        b.forward()
        b.backward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        b.forward()
        b.backward()
    for src in (eager, other):
        if src is other:
            other.backward()
        for key in ("x", "v", "q", "router", "w1", "w2", "dn"):
            getattr(b, key).copy_(getattr(src, key))
        for t in (b.drouter, b.dw1, b.dw2, b.dq, b.out):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for key, got in b.grads().items():
            assert torch.equal(got, src.grads()[key]), key
        assert torch.equal(b.out, src.out) and torch.equal(b.loss, src.loss)


def test_calls_at_once_on_two_streams(dfm):
    """Each with outputs and workspaces of its own: the same bits as alone."""
    blocks, alone = [Block(dfm, 21), Block(dfm, 22)], [Block(dfm, 21), Block(dfm, 22)]
    for b in alone:
        b.forward()
        b.backward()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for b, s in zip(blocks, streams):
            with torch.cuda.stream(s):
                b.forward()
                b.backward()
    torch.cuda.synchronize()
    for b, want in zip(blocks, alone):
        for key, got in b.grads().items():
            assert torch.equal(got, want.grads()[key]), key
        assert torch.equal(b.out, want.out)


def test_calls_run_on_torchs_current_stream(dfm):
    """Between a producer and a consumer of the same stream, without synchronising."""
    T, H = 2048, 4096
    s = torch.cuda.Stream()
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    w = torch.eye(H, device="cuda").to(torch.bfloat16)
    n, y = torch.empty_like(x), torch.empty_like(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(10):
            big = big @ big * 1e-4  # keeps the stream busy
        x.fill_(2.0)
        dfm.block_norm(None, x, "bf16", T, H, n=n)
        dfm.matmul(n, w, "bf16", T, H, H, y, "bf16")
        got = y.clone()
    s.synchronize()
    assert bool((got == 1).all())


def test_arrays_of_several_devices_are_refused(dfm):
    class Elsewhere:
        def get_device(self):
            return 1

        def data_ptr(self):
            return 1 << 20
    x = torch.zeros(8, 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(dfm.DfMoeError, match="different devices"):
        dfm.matmul(x, Elsewhere(), "bf16", 8, 8, 8, x, "bf16")
