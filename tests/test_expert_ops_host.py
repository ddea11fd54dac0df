"""Refusals of the expert-path operators (no GPU needed): every bad argument is
an error code and a message before a device is touched. Addresses are made up
and never followed."""
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


PERMUTE = dict(ids=A, T=4, k=2, E=8, x=A, dtype="bf16", H=64, rows=A, offs=A, pos=A, src=A)


@pytest.mark.parametrize("change, code, word", [
    (dict(T=-1), -1, "negative"), (dict(k=0), -1, "k must"), (dict(k=33), -1, "k must"),
    (dict(E=0), -1, "E must"), (dict(E=1025), -1, "E must"), (dict(H=0), -1, "H must"),
    (dict(H=262145), -1, "H must"), (dict(T=1 << 31, k=1), -5, "assignments"),
    (dict(T=1 << 30, k=2), -5, "assignments"), (dict(dtype=4), -1, "dtype"),
    (dict(dtype="f64"), -1, "dtype"), (dict(ldx=63), -1, "ldx"), (dict(ldr=1), -1, "ldr"),
    (dict(ids=None), -1, "required"), (dict(x=None), -1, "required"), (dict(rows=None), -1, "required"),
    (dict(offs=None), -1, "offs"), (dict(pos=None), -1, "required"), (dict(src=None), -1, "required"),
    (dict(x=A + 1), -1, "aligned"), (dict(rows=A + 1), -1, "aligned"), (dict(ids=A + 2), -1, "aligned"),
    (dict(offs=A + 2), -1, "aligned"), (dict(n_scales=-1), -1, "n_scales"),
    (dict(n_scales=2), -1, "rows_scales"), (dict(n_scales=2, scales=A, rows_scales=A, ld_scales=1), -1, "ld_scales"),
    (dict(n_scales=2, scales=A + 1, rows_scales=A), -1, "aligned"),
    (dict(T=65537, k=1), -1, "workspace"), (dict(T=65537, k=1, workspace=A, workspace_bytes=16), -1, "workspace"),
    (dict(T=65537, k=1, workspace=A + 1, workspace_bytes=1 << 22), -1, "workspace"),
])
def test_permute_refusals(dfm, change, code, word):
    refused(dfm, dfm.permute, code, word, **dict(PERMUTE, **change))


def test_permute_workspace_sizes(dfm):
    assert dfm.permute_workspace(4096, 16, 1024) == 0
    assert dfm.permute_workspace(65537, 1, 8) > 0
    # the largest call fits the 4 MiB that the header names
    assert dfm.permute_workspace((1 << 31) - 1, 1, 1024) == 4 << 20
    assert dfm.permute_workspace(0, 1, 8) == dfm.permute_workspace(1, 0, 8) == 0


UNPERMUTE = dict(rows=A, dtype="f32", n_rows=8, pos=A, weights=A, T=4, k=2, H=64, y=A)


@pytest.mark.parametrize("change, code, word", [
    (dict(T=-1), -1, "negative"), (dict(k=0), -1, "k must"), (dict(H=0), -1, "H must"),
    (dict(dtype="e4m3"), -1, "dtype"), (dict(n_rows=-1), -1, "n_rows"), (dict(ldr=63), -1, "distance"),
    (dict(ldy=63), -1, "distance"), (dict(rows=None), -1, "required"), (dict(pos=None), -1, "required"),
    (dict(weights=None), -1, "weights"), (dict(y=None), -1, "required"), (dict(y=A + 2), -1, "aligned"),
    (dict(pos=A + 1), -1, "aligned"), (dict(T=(1 << 31) - 1, k=1, H=262144), -5, "too large"),
])
def test_unpermute_refusals(dfm, change, code, word):
    kw = dict(UNPERMUTE, **change)
    refused(dfm, dfm.unpermute, code, word, **kw)
    if "weights" not in change:
        kw.pop("weights")
        kw["drows"], kw["dx"] = kw.pop("rows"), kw.pop("y")
        kw["ldx"] = kw.pop("ldy", 0)
        refused(dfm, dfm.permute_grad, code, word, **kw)


GRAD = dict(dy=A, rows=A, dtype="bf16", n_rows=8, pos=A, weights=A, T=4, k=2, H=64, drows=A, dweights=A)


@pytest.mark.parametrize("change, code, word", [
    (dict(T=-1), -1, "negative"), (dict(k=33), -1, "k must"), (dict(dtype="e4m3"), -1, "dtype"),
    (dict(lddy=1), -1, "lddy"), (dict(ldr=1), -1, "ldr"), (dict(lddr=1), -1, "lddr"),
    (dict(dy=None), -1, "required"), (dict(rows=None), -1, "required"), (dict(drows=None), -1, "required"),
    (dict(weights=None), -1, "required"), (dict(dweights=None), -1, "required"),
    (dict(drows=A + 1), -1, "aligned"), (dict(n_rows=-2), -1, "n_rows"),
])
def test_unpermute_grad_refusals(dfm, change, code, word):
    refused(dfm, dfm.unpermute_grad, code, word, **dict(GRAD, **change))


QUANT = dict(x=A, dtype="bf16", M=4, K=256, codes=A, scales=A)


@pytest.mark.parametrize("change, code, word", [
    (dict(M=-1), -1, "negative"), (dict(K=0), -1, "K must"), (dict(K=262145), -1, "K must"),
    (dict(dtype="e4m3"), -1, "dtype"), (dict(ldx=255), -1, "ldx"), (dict(ldc=255), -1, "ldc"),
    (dict(lds=1), -1, "lds"), (dict(x=None), -1, "required"), (dict(codes=None), -1, "required"),
    (dict(scales=None), -1, "required"), (dict(x=A + 1), -1, "aligned"), (dict(scales=A + 2), -1, "aligned"),
    (dict(M=1 << 30), -5, "2^31"),
])
def test_quantize_refusals(dfm, change, code, word):
    refused(dfm, dfm.fp8_quantize, code, word, **dict(QUANT, **change))


MATMUL = dict(x=A, xs=A, w=A, ws=A, offs=A, G=4, M=64, N=128, K=256, y=A, dtype="bf16")


@pytest.mark.parametrize("change, code, word", [
    (dict(M=-1), -1, "negative"), (dict(M=1 << 31), -5, "M must"), (dict(N=0), -1, "N must"),
    (dict(K=0), -1, "K must"), (dict(N=262145), -1, "N must"), (dict(G=0), -1, "G must"),
    (dict(G=1025), -1, "G must"), (dict(offs=None), -1, "offs"), (dict(dtype="e4m3"), -1, "dtype"),
    (dict(K=250), -1, "ldx"), (dict(ldx=264), -1, "ldx"), (dict(ldw=264), -1, "ldw"),
    (dict(ldw=240), -1, "ldw"), (dict(N=100, transposed=True), -1, "ldw"), (dict(ldxs=1), -1, "ldxs"),
    (dict(ldy=127), -1, "ldy"), (dict(x=None), -1, "required"), (dict(xs=None), -1, "required"),
    (dict(w=None), -1, "required"), (dict(ws=None), -1, "required"), (dict(y=None), -1, "required"),
    (dict(x=A + 8), -1, "16-byte"), (dict(w=A + 8), -1, "16-byte"), (dict(y=A + 1), -1, "aligned"),
    (dict(xs=A + 2), -1, "aligned"), (dict(offs=A + 1), -1, "aligned"), (dict(status=A + 1), -1, "aligned"),
    (dict(ldx=1 << 39), -5, "too large"), (dict(ldw=1 << 34), -5, "too large"),
])
def test_matmul_refusals(dfm, change, code, word):
    refused(dfm, dfm.fp8_matmul, code, word, **dict(MATMUL, **change))


def test_host_arrays_are_refused(dfm):
    import numpy as np
    import torch
    for bad in (torch.zeros(8), np.zeros(8, np.float32)):
        refused(dfm, dfm.fp8_quantize, -1, "device memory", **dict(QUANT, x=bad))


def test_without_a_device_the_call_says_so(dfm):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is here")
    refused(dfm, dfm.fp8_quantize, -3, "no CUDA device", **QUANT)


def test_empty_calls_need_no_device(dfm):
    dfm.fp8_quantize(None, "bf16", 0, 128, None, None)
    dfm.fp8_matmul(None, None, None, None, None, 1, 0, 128, 128, None, "bf16")
    dfm.unpermute(None, "bf16", 0, None, None, 0, 2, 64, None)
    dfm.permute_grad(None, "bf16", 0, None, 0, 2, 64, None)
    dfm.unpermute_grad(None, None, "bf16", 0, None, None, 0, 2, 64, None, None)


class OnDevice0:
    """Stands for a torch tensor on device 0: an address, never followed."""

    def get_device(self):
        return 0

    def data_ptr(self):
        return A


EVERY_CALL = [
    ("permute", PERMUTE), ("permute_grad", dict(drows=A, dtype="f32", n_rows=8, pos=A, T=4, k=2, H=64, dx=A)),
    ("unpermute", UNPERMUTE), ("unpermute_grad", GRAD), ("fp8_quantize", QUANT), ("fp8_matmul", MATMUL),
]


@pytest.mark.parametrize("name, kw", EVERY_CALL)
def test_a_call_without_a_stream_runs_on_the_current_one(dfm, monkeypatch, name, kw):
    """Tensors: the stream that torch has current on their device. Raw
    addresses only: the default stream. A stream that is given is taken."""
    import torch
    binding, seen = dfm.binding, []
    monkeypatch.setattr(binding._c, "df_moe_" + name, lambda *a: seen.append(a[-1]) or 0)
    monkeypatch.setattr(binding, "_torch_stream", binding._find_torch_stream)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0x5000 + dev)
    call = getattr(dfm, name)
    tensors = {key: OnDevice0() if v == A else v for key, v in kw.items()}
    call(**tensors)
    call(**kw)
    call(**dict(tensors, stream=0x77))
    call(**dict(tensors, stream=0))
    assert seen == [0x5000, None, 0x77, 0]


ROW_WORD_TEST = r"""
#include <cstdint>
#include <cstdio>
#include "rowword.h"
// Every read of an array, checked: n values, the first of them at address `at`
// (in values), where words of four start at multiples of four.
struct Checked {
  int at, n;
  void seen(int64_t i) const { if (i < 0 || i >= n) { std::printf("read of value %d of %d\n", (int)i, n); throw 1; } }
  dfm::Four<uint16_t> four(int64_t i) const {
    dfm::Four<uint16_t> r;
    if ((at + i) & 3) { std::printf("word %d not aligned\n", (int)(at + i)); throw 1; }
    for (int u = 0; u < 4; ++u) { seen(i + u); r.v[u] = (uint16_t)(100 + i + u); }
    return r;
  }
  uint16_t one(int64_t i) const { seen(i); return (uint16_t)(100 + i); }
};
int main() {
  for (int at = 8; at < 12; ++at)
    for (int n = 1; n < 40; ++n)
      for (int w = 0; w < 60; w += 4) {
        const dfm::Four<uint16_t> r = dfm::array_four<uint16_t>(Checked{at, n}, w - at, n);
        for (int u = 0; u < 4; ++u) {
          const int i = w - at + u;
          if (r.v[u] != (i >= 0 && i < n ? 100 + i : 0)) { std::printf("value %d of %d\n", i, n); return 1; }
        }
      }
  return 0;
}
"""


def test_words_of_unaligned_rows_read_nothing_beside_the_array(tmp_path):
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    (tmp_path / "t.cpp").write_text(ROW_WORD_TEST)
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(root, "mxfp4_routed_expert_top_gb300", "csrc"), "-o",
                    str(tmp_path / "t"), str(tmp_path / "t.cpp")], check=True)
    r = subprocess.run([str(tmp_path / "t")], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_matmul_refuses_a_row_distance_whose_product_overflows(dfm):
    refused(dfm, dfm.fp8_matmul, -5, "too large", **dict(MATMUL, ldw=1 << 62))
    refused(dfm, dfm.fp8_matmul, -5, "too large", **dict(MATMUL, N=256, ldw=1 << 56))


@pytest.mark.parametrize("name, kw", EVERY_CALL[:4] + EVERY_CALL[5:])
def test_sizes_that_32_bits_would_cut_are_refused(dfm, name, kw):
    """2^32 + 2 is not 2."""
    for size in ("k", "E", "n_scales", "G"):
        if size in kw or (size == "n_scales" and name == "permute"):
            for v in (1 << 31, (1 << 32) + 2, (1 << 64) + 2):
                refused(dfm, getattr(dfm, name), -1, "32 bits", **dict(kw, **{size: v}))
    assert dfm.permute_workspace(70000, (1 << 32) + 2, 8) == dfm.permute_workspace(70000, 2, (1 << 32) + 8) == 0


def test_permute_refuses_a_negative_workspace_size(dfm):
    refused(dfm, dfm.permute, -1, "workspace_bytes", **dict(PERMUTE, T=65537, k=1, workspace=A, workspace_bytes=-1))
