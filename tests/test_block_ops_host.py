"""Refusals of the operators around the routed experts (no GPU needed): every bad
argument is an error code and a message before a device is touched. Addresses
are made up and never followed."""
import pytest


@pytest.fixture(scope="module")
def dfm():
    import __graft_entry__
    __graft_entry__.build()
    import mxfp4_routed_expert_top_gb300 as m
    return m


A = 1 << 20  # an aligned address


def refused(dfm, f, code, word, **kw):
    with pytest.raises(dfm.DfMoeError) as ei:
        f(**kw)
    assert ei.value.code == code, str(ei.value)
    assert word in str(ei.value), str(ei.value)


MATMUL = dict(x=A, w=A, dtype="bf16", M=64, N=128, K=256, y=A, out_dtype="f32")


@pytest.mark.parametrize("change, code, word", [
    (dict(M=-1), -1, "negative"), (dict(M=(1 << 31) - 256), -5, "M must"), (dict(N=0), -1, "N must"), (dict(K=0), -1, "K must"),
    (dict(N=262145), -1, "N must"), (dict(K=262145), -1, "K must"), (dict(dtype="f32"), -1, "dtype"),
    (dict(dtype="e4m3"), -1, "dtype"), (dict(dtype="f64"), -1, "dtype"), (dict(out_dtype="f16"), -1, "out_dtype"),
    (dict(dtype="f16", out_dtype="bf16"), -1, "out_dtype"), (dict(act="tanh"), -1, "act"), (dict(act=None), -1, "act"),
    (dict(K=250), -1, "multiple of 8"), (dict(ldx=264, K=265), -1, "multiple of 8"), (dict(ldx=248), -1, "multiple of 8"),
    (dict(ldw=260), -1, "multiple of 8"), (dict(ldw=248), -1, "multiple of 8"), (dict(ldy=127), -1, "ldy"),
    (dict(residual=A, ldr=127), -1, "residual"), (dict(pre=A, ldp=127), -1, "pre"),
    (dict(pre=A, ldp=255, act="swiglu"), -1, "pre"), (dict(x=None), -1, "required"), (dict(w=None), -1, "required"),
    (dict(y=None), -1, "required"), (dict(x=A + 8), -1, "16-byte"), (dict(w=A + 2), -1, "16-byte"),
    (dict(y=A + 2), -1, "aligned"), (dict(residual=A + 2), -1, "aligned"), (dict(pre=A + 1), -1, "aligned"),
    (dict(bias=A + 1), -1, "aligned"), (dict(status=A + 2), -1, "aligned"), (dict(ldx=1 << 39), -5, "too large"),
    (dict(ldw=1 << 62), -5, "too large"), (dict(M=1 << 64), -1, "64 bits"), (dict(ldx=(1 << 64) + 256), -1, "64 bits"),
])
def test_matmul_refusals(dfm, change, code, word):
    refused(dfm, dfm.matmul, code, word, **dict(MATMUL, **change))


GRAD = dict(dy=A, x=A, w=A, dtype="bf16", M=64, N=128, K=256, dx=A, dw=A, dbias=A, act="swiglu", pre=A, dz=A)


@pytest.mark.parametrize("change, code, word", [
    (dict(M=-1), -1, "negative"), (dict(M=1 << 31), -5, "M must"), (dict(N=0), -1, "N must"), (dict(K=1 << 20), -1, "K must"),
    (dict(dtype="f32"), -1, "dtype"), (dict(grad_dtype="f16"), -1, "grad_dtype"), (dict(grad_dtype="e4m3"), -1, "grad_dtype"),
    (dict(act="relu6"), -1, "act"), (dict(dx=None, dw=None, dbias=None, act="none"), -1, "none of"),
    (dict(pre=None), -1, "pre and dz"), (dict(dz=None), -1, "pre and dz"), (dict(ldp=255), -1, "pre"),
    (dict(lddz=255), -1, "dz"), (dict(lddz=260), -1, "multiple of 8"), (dict(dz=A + 2), -1, "16-byte"),
    (dict(N=127, lddz=255), -1, "multiple of 8"), (dict(N=127), -1, "multiple of 8"),
    (dict(lddy=127), -1, "dy"), (dict(act="none", lddy=132), -1, "multiple of 8"), (dict(act="none", dy=A + 2), -1, "16-byte"),
    (dict(act="none", dx=None, dw=None, lddy=127), -1, "dy"), (dict(dy=None), -1, "required"), (dict(x=None), -1, "required"),
    (dict(w=None), -1, "required"), (dict(x=A + 8), -1, "16-byte"), (dict(w=A + 8), -1, "16-byte"),
    (dict(K=250), -1, "multiple of 8"), (dict(lddx=255), -1, "dx"), (dict(lddw=255), -1, "dw"), (dict(dx=A + 1), -1, "dx"),
    (dict(dw=A + 2), -1, "dw"), (dict(dbias=A + 2), -1, "aligned"), (dict(status=A + 1), -1, "aligned"),
    (dict(lddz=1 << 39), -5, "too large"), (dict(lddw=1 << 64), -1, "64 bits"),
])
def test_matmul_grad_refusals(dfm, change, code, word):
    refused(dfm, dfm.matmul_grad, code, word, **dict(GRAD, **change))


NORM = dict(u=A, residual=A, dtype="bf16", T=4, H=64, h=A, n=A, post=True, post_weight=A, gate=A, gate_kind="channel",
            pre_weight=A)
NORM_GRAD = dict(dh=A, dn=A, u=A, h=A, dtype="bf16", T=4, H=64, du=A, dresidual=A, post=True, post_weight=A, dpost_weight=A,
                 gate=A, gate_kind="channel", dgate=A, pre_weight=A, dpre_weight=A, workspace=A, workspace_bytes=1 << 30)


@pytest.mark.parametrize("change, code, word", [
    (dict(T=-1), -1, "negative"), (dict(T=1 << 31), -5, "T must"), (dict(H=0), -1, "H must"), (dict(H=32769), -1, "H must"),
    (dict(dtype="e4m3"), -1, "dtype"), (dict(weight_dtype="f16"), -1, "weight_dtype"), (dict(eps=0.0), -1, "eps"),
    (dict(eps=-1e-6), -1, "eps"), (dict(eps=float("nan")), -1, "eps"), (dict(eps=float("inf")), -1, "eps"),
    (dict(gate_kind="row"), -1, "gate_kind"), (dict(gate=None), -1, "gate"), (dict(gate=A + 2), -1, "aligned"),
    (dict(gate_kind="token", gate=A + 2), -1, "aligned"), (dict(gate_kind="full", gate=A + 1), -1, "gate"),
    (dict(gate_kind="full", ldg=63), -1, "gate"), (dict(post_weight=A + 2), -1, "aligned"),
    (dict(pre_weight=A + 2), -1, "aligned"), (dict(T=1 << 64), -1, "64 bits"),
])
def test_norm_refusals(dfm, change, code, word):
    refused(dfm, dfm.block_norm, code, word, **dict(NORM, **change))
    refused(dfm, dfm.block_norm_grad, code, word, **dict(NORM_GRAD, **change))


@pytest.mark.parametrize("change, code, word", [
    (dict(ldu=63), -1, "u"), (dict(ldr=63), -1, "residual"), (dict(ldh=1), -1, "h"), (dict(ldn=-1), -1, "n"),
    (dict(u=A + 1), -1, "u"), (dict(residual=A + 1), -1, "residual"), (dict(h=A + 1), -1, "h"), (dict(n=A + 1), -1, "n"),
    (dict(u=None, residual=None), -1, "required"), (dict(h=None, n=None), -1, "required"), (dict(u=None), -1, "u"),
    (dict(u=None, gate_kind="none", gate=None), -1, "needs u"), (dict(post=False), -1, "post"),
])
def test_block_norm_refusals(dfm, change, code, word):
    refused(dfm, dfm.block_norm, code, word, **dict(NORM, **change))


@pytest.mark.parametrize("change, code, word", [
    (dict(lddh=63), -1, "dh"), (dict(lddn=63), -1, "dn"), (dict(ldu=63), -1, "u"), (dict(ldh=63), -1, "h"),
    (dict(lddu=63), -1, "du"), (dict(lddr=63), -1, "dresidual"), (dict(gate_kind="full", lddg=63), -1, "dgate"),
    (dict(dh=None, dn=None), -1, "required"), (dict(h=None), -1, "needs h"), (dict(u=None), -1, "need u"),
    (dict(dn=None), -1, "need dn"), (dict(dn=None, pre_weight=None), -1, "need dn"),
    (dict(du=None, dresidual=None, dpost_weight=None, dgate=None, dpre_weight=None), -1, "no gradient"),
    (dict(post=False), -1, "post"), (dict(post=False, post_weight=None), -1, "post"),
    (dict(gate_kind="none"), -1, "dgate"), (dict(workspace=None), -1, "workspace"), (dict(workspace_bytes=64), -1, "workspace"),
    (dict(workspace=A + 4), -1, "workspace"), (dict(workspace_bytes=-1), -1, "workspace"), (dict(dpost_weight=A + 2), -1, "aligned"),
    (dict(dgate=A + 2), -1, "aligned"), (dict(dpre_weight=A + 1), -1, "aligned"),
])
def test_block_norm_grad_refusals(dfm, change, code, word):
    refused(dfm, dfm.block_norm_grad, code, word, **dict(NORM_GRAD, **change))


def test_norm_workspace_sizes(dfm):
    small = dfm.block_norm_grad_workspace(1, 64)
    assert 0 < small <= dfm.block_norm_grad_workspace(1 << 20, 64)
    assert dfm.block_norm_grad_workspace(1 << 31 - 1, 32768) > 0
    for bad in ((0, 64), (-1, 64), (1, 0), (1, 32769), (1 << 31, 64), (1 << 65, 64)):
        assert dfm.block_norm_grad_workspace(*bad) == 0


BALANCE = dict(logits=A, dtype="f32", T=8, E=16, ids=A, k=2, loss=A, counts=A, tokens=A, workspace=A, workspace_bytes=1 << 30)
BALANCE_GRAD = dict(dloss=A, logits=A, dtype="f32", T=8, E=16, ids=A, k=2, counts=A, tokens=A, dlogits=A, weights=A, dweights=A)


@pytest.mark.parametrize("change, code, word", [
    (dict(T=-1), -1, "negative"), (dict(T=1 << 31), -5, "T * k"), (dict(E=0), -1, "E must"), (dict(E=1025), -1, "E must"),
    (dict(k=0), -1, "k must"), (dict(k=33), -1, "k must"), (dict(S=0), -1, "S must"), (dict(S=(1 << 20) + 1, offs=A), -5, "S must"),
    (dict(S=2), -1, "offs"), (dict(score="tanh"), -1, "score"), (dict(dtype="e4m3"), -1, "dtype"),
    (dict(coef=float("inf")), -1, "finite"), (dict(z_coef=float("nan")), -1, "finite"), (dict(ldl=15), -1, "ldl"),
    (dict(logits=None), -1, "required"), (dict(logits=A + 2), -1, "aligned"), (dict(counts=A + 2), -1, "aligned"),
    (dict(tokens=A + 1), -1, "aligned"), (dict(ids=A + 2), -1, "aligned"), (dict(offs=A + 2), -1, "aligned"),
    (dict(counts=None), -1, "required"), (dict(tokens=None), -1, "required"), (dict(E=(1 << 32) + 2), -1, "32 bits"),
    (dict(k=(1 << 32) + 2), -1, "32 bits"), (dict(T=1 << 64), -1, "64 bits"),
])
def test_balance_refusals(dfm, change, code, word):
    refused(dfm, dfm.balance_loss, code, word, **dict(BALANCE, **change))
    refused(dfm, dfm.balance_loss_grad, code, word, **dict(BALANCE_GRAD, **change))


@pytest.mark.parametrize("name, change, code, word", [
    ("balance_loss", dict(loss=None), -1, "required"), ("balance_loss", dict(ids=None), -1, "required"),
    ("balance_loss", dict(workspace=None), -1, "workspace"), ("balance_loss", dict(workspace_bytes=32), -1, "workspace"),
    ("balance_loss", dict(workspace=A + 8), -1, "workspace"), ("balance_loss", dict(probs=A + 2), -1, "aligned"),
    ("balance_loss", dict(status=A + 2), -1, "aligned"), ("balance_loss", dict(workspace_bytes=-5), -1, "workspace"),
    ("balance_loss_grad", dict(dloss=None), -1, "required"), ("balance_loss_grad", dict(dlogits=None), -1, "required"),
    ("balance_loss_grad", dict(lddl=15), -1, "lddl"), ("balance_loss_grad", dict(weights=None), -1, "together"),
    ("balance_loss_grad", dict(dweights=None), -1, "together"), ("balance_loss_grad", dict(ids=None), -1, "together"),
    ("balance_loss_grad", dict(dlogits=A + 2), -1, "aligned"), ("balance_loss_grad", dict(weights=A + 2), -1, "aligned"),
])
def test_balance_refusals_of_one(dfm, name, change, code, word):
    refused(dfm, getattr(dfm, name), code, word, **dict(BALANCE if name == "balance_loss" else BALANCE_GRAD, **change))


def test_balance_workspace_sizes(dfm):
    assert 0 < dfm.balance_loss_workspace(1, 8) <= dfm.balance_loss_workspace(1, 8, 5)
    for bad in ((0, 8), (1, 0), (1, 1025), (1, 8, 0), (1 << 31, 8), (1, 8, (1 << 20) + 1), (1, 1 << 40), (1 << 65, 8)):
        assert dfm.balance_loss_workspace(*bad) == 0


def test_give_up_hook_refuses_unknown_roles(dfm):
    for role in (-1, 4):
        refused(dfm, dfm.test_matmul_give_up, -1, "role", role=role)


def test_empty_calls_need_no_device(dfm):
    dfm.matmul(None, None, "bf16", 0, 128, 128, None, "bf16")
    dfm.matmul_grad(None, None, None, "bf16", 0, 128, 128, dx=A)
    dfm.block_norm(None, None, "bf16", 0, 64)
    dfm.block_norm_grad(None, None, None, None, "bf16", 0, 64, du=A)
    dfm.balance_loss_grad(None, None, "f32", 0, 8, None, 2, None, None, None)


EVERY_CALL = [("matmul", MATMUL), ("matmul_grad", GRAD), ("block_norm", NORM), ("block_norm_grad", NORM_GRAD),
              ("balance_loss", BALANCE), ("balance_loss_grad", BALANCE_GRAD)]


@pytest.mark.parametrize("name, kw", EVERY_CALL)
def test_host_arrays_and_missing_devices_are_refused(dfm, name, kw):
    import torch
    for key, v in kw.items():
        if v == A:
            refused(dfm, getattr(dfm, name), -1, "device memory", **dict(kw, **{key: torch.zeros(8)}))
    if not torch.cuda.is_available():
        refused(dfm, getattr(dfm, name), -3, "no CUDA device", **kw)


class OnDevice0:
    """Stands for a torch tensor on device 0: an address, never followed."""

    def get_device(self):
        return 0

    def data_ptr(self):
        return A


@pytest.mark.parametrize("name, kw", EVERY_CALL)
def test_a_call_without_a_stream_runs_on_the_current_one(dfm, monkeypatch, name, kw):
    """The stream is the last of the values that a call packs."""
    import struct
    import torch
    binding, seen = dfm.binding, []
    monkeypatch.setattr(binding._c, "df_moe_packed", lambda call, args: seen.append(struct.unpack("q", args[-8:])[0]) or 0)
    monkeypatch.setattr(binding, "_torch_stream", binding._find_torch_stream)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0x5000 + dev)
    call = getattr(dfm, name)
    tensors = {key: OnDevice0() if v == A else v for key, v in kw.items()}
    call(**tensors)
    call(**kw)
    call(**dict(tensors, stream=0x77))
    assert seen == [0x5000, 0, 0x77]


def test_packed_calls_are_the_calls(dfm):
    """Every argument in its place: both ways give the same code and message."""
    import ctypes
    import struct
    L = dfm.lib()
    vp, i32, i64, f32, ci = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_int
    kinds = {  # as the header has them
        "matmul": [ci, vp, i64, vp, i64, i32, i64, i64, i64, vp, i32, vp, i64, vp, i64, vp, i32, i64, vp, vp],
        "matmul_grad": [ci, vp, i64, vp, i64, vp, i64, i32, i64, i64, i64, i32, vp, i64, vp, i64, vp, i64, vp, i64, vp, i32, vp, vp],
        "block_norm": [ci, vp, i64, i32, vp, i32, vp, i64, vp, i64, f32, vp, f32, i64, i64, i32, i32, vp, i64, vp, i64, vp],
        "block_norm_grad": [ci, vp, i64, vp, i64, vp, i64, vp, i64, i32, vp, i32, vp, i64, f32, vp, f32, i64, i64, i32, i32, vp, i64,
                            vp, i64, vp, vp, i64, vp, vp, ctypes.c_size_t, vp],
        "balance_loss": [ci, vp, i32, i64, vp, i64, i32, i32, vp, i64, vp, i32, f32, f32, vp, vp, vp, vp, vp, ctypes.c_size_t, vp, vp],
        "balance_loss_grad": [ci, vp, vp, i32, i64, vp, i64, i32, i32, vp, i64, vp, i32, f32, f32, vp, vp, vp, vp, vp, i64, vp],
    }
    values = {vp: (0, A, A + 1), i64: (0, 8, 64, -1, 1 << 40), i32: (0, 1, 2, 9), f32: (0.0, 1.0, 1e-6, float("nan")), ci: (0,),
              ctypes.c_size_t: (0, 1 << 30)}
    import random
    rng = random.Random(0)
    for call, (name, types) in enumerate(kinds.items()):
        f = getattr(L, "df_moe_" + name)
        f.argtypes = types
        for _ in range(3000):
            args = [rng.choice(values[t]) for t in types]
            args[0] = 1 << 20  # no such device: nothing is launched
            block = b"".join(struct.pack("d" if t is f32 else "q", v) for t, v in zip(types, args))
            want = f(*args)
            message = L.df_moe_last_error(None)
            assert L.df_moe_packed(call, block) == want
            if want:
                assert L.df_moe_last_error(None) == message
    assert L.df_moe_packed(6, b"") == -1 and L.df_moe_packed(-1, b"") == -1


class Elements(OnDevice0):
    """The same with elements of a size."""

    def __init__(self, size):
        self.size = size

    def element_size(self):
        return self.size


# The calls, and the bytes of an element of every array: 16-bit operands, fp32
# where a call names no other type.
ELEMENTS = [
    ("matmul", MATMUL, dict(x=2, w=2, y=4, bias=2, residual=4, pre=2, status=4)),
    ("matmul", dict(MATMUL, out_dtype="bf16"), dict(x=2, w=2, y=2, bias=2, residual=2, pre=2, status=4)),
    ("matmul_grad", GRAD, dict(dy=2, x=2, w=2, dx=2, dw=4, dbias=4, pre=2, dz=2, status=4)),
    ("matmul_grad", dict(GRAD, grad_dtype="bf16"), dict(dy=2, x=2, w=2, dx=2, dw=2, dbias=2, pre=2, dz=2, status=4)),
    ("block_norm", NORM, dict(u=2, residual=2, h=2, n=2, post_weight=4, gate=4, pre_weight=4)),
    ("block_norm", dict(NORM, weight_dtype="bf16"), dict(u=2, residual=2, h=2, n=2, post_weight=2, gate=2, pre_weight=2)),
    ("block_norm", dict(NORM, gate_kind="token", weight_dtype="bf16"), dict(u=2, gate=4, pre_weight=2)),
    ("block_norm", dict(NORM, gate_kind="full"), dict(u=2, gate=2, pre_weight=4)),
    ("block_norm", dict(NORM, u=None), dict(residual=2, h=2, n=2, pre_weight=4)),
    ("block_norm_grad", NORM_GRAD, dict(dh=2, dn=2, u=2, h=2, du=2, dresidual=2, post_weight=4, dpost_weight=4, gate=4, dgate=4,
                                        pre_weight=4, dpre_weight=4)),
    ("block_norm_grad", dict(NORM_GRAD, weight_dtype="bf16"), dict(post_weight=2, dpost_weight=4, gate=2, dgate=4, pre_weight=2,
                                                                   dpre_weight=4)),
    ("block_norm_grad", dict(NORM_GRAD, gate_kind="token"), dict(dh=2, gate=4, dgate=4)),
    ("block_norm_grad", dict(NORM_GRAD, gate_kind="full"), dict(dh=2, gate=2, dgate=2)),
    ("balance_loss", BALANCE, dict(logits=4, ids=4, loss=4, counts=4, tokens=4, probs=4, offs=4, mask=1, status=4)),
    ("balance_loss", dict(BALANCE, dtype="f16"), dict(logits=2, ids=4)),
    ("balance_loss_grad", BALANCE_GRAD, dict(dloss=4, logits=4, ids=4, counts=4, tokens=4, dlogits=4, offs=4, mask=1, weights=4,
                                             dweights=4)),
    ("balance_loss_grad", dict(BALANCE_GRAD, dtype="bf16"), dict(dloss=4, logits=2, dlogits=2)),
]


@pytest.mark.parametrize("name, kw, elements", ELEMENTS)
@pytest.mark.parametrize("real", [False, True])
def test_arrays_of_another_types_size_are_refused(dfm, monkeypatch, name, kw, elements, real):
    """A named type wider than the tensor's, a default among them, would be read
    and written past its end. A workspace's elements are not looked at."""
    import torch
    binding, seen = dfm.binding, []
    monkeypatch.setattr(binding._c, "df_moe_packed", lambda call, args: seen.append(args) or 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0x5000)
    monkeypatch.setattr(binding, "_torch_stream", binding._find_torch_stream)
    types = {1: torch.bool, 2: torch.bfloat16, 4: torch.float32, 8: torch.int64}
    if real:  # torch's tensors, which stand for some on device 0
        monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
        monkeypatch.setattr(binding, "_get_device", lambda a: 0 if torch.is_tensor(a) else binding._find_tensor_calls(a))
        monkeypatch.setattr(binding, "_element_size", torch.Tensor.element_size)
        monkeypatch.setattr(binding, "_data_ptr", torch.Tensor.data_ptr)
    make = (lambda n: torch.zeros(1, dtype=types[n])) if real else Elements
    arrays = {key: make(n) for key, n in elements.items()}
    rest = {key: None if key not in elements and key not in ("workspace",) and v == A else v for key, v in kw.items()}
    if "workspace" in kw:
        rest["workspace"] = make(1)
    getattr(dfm, name)(**dict(rest, **arrays))
    assert len(seen) == 1
    for key, n in elements.items():
        for other in {1, 2, 4, 8} - {n} - ({8} if key == "status" else set()):
            refused(dfm, getattr(dfm, name), -1, "%s has elements of %d bytes" % (key, other),
                    **dict(rest, **dict(arrays, **{key: make(other)})))
    assert len(seen) == 1


@pytest.mark.parametrize("v", [-(1 << 32) + 8, -(1 << 31) - 1, -(1 << 63)])
def test_sizes_that_32_bits_would_cut_are_refused(dfm, v):
    """-2^32 + 8 is not 8, and without rows neither."""
    for T in (8, 0):
        for key in ("E", "k"):
            refused(dfm, dfm.balance_loss, -1, "32 bits", **dict(BALANCE, T=T, **{key: v}))
            refused(dfm, dfm.balance_loss_grad, -1, "32 bits", **dict(BALANCE_GRAD, T=T, **{key: v}))
    assert dfm.balance_loss_workspace(64, v, 1) == 0


def test_packed_integers_that_do_not_fit_are_refused(dfm):
    import struct
    L = dfm.lib()
    kinds = {0: "ipqpqiqqqpipqpqpiqpp", 1: "ipqpqpqiqqqipqpqpqpqpipp", 2: "ipqipipqpqfpfqqiipqpqp",
             3: "ipqpqpqpqipipqfpfqqiipqpqppqppzp", 4: "ipiqpqiipqpiffpppppzpp", 5: "ippiqpqiipqpiffpppppqp"}
    for call, types in kinds.items():
        args = [0.0 if t == "f" else 0 for t in types]
        args[0] = 1 << 20  # no such device
        layout = "".join("d" if t == "f" else "q" for t in types)
        for i, t in enumerate(types):
            for v in ((1 << 31, 1 << 32, (1 << 32) + 2, -(1 << 32) + 2, -(1 << 31) - 1) if t == "i" else (-1, -(1 << 63)) if t == "z" else ()):
                assert L.df_moe_packed(call, struct.pack(layout, *(args[:i] + [v] + args[i + 1:]))) == -1
                assert b"does not fit" in L.df_moe_last_error(None), (call, i, v)
        L.df_moe_packed(call, struct.pack(layout, *args))
        assert b"does not fit" not in (L.df_moe_last_error(None) or b"")
