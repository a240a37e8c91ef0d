"""Host side of the operators between a model's parameters and the points: the
C structure's layout, and the checks that need no GPU."""
import ctypes
import os
import shutil
import subprocess

import pytest

from conftest import ROOT


def _edd():
    import __graft_entry__
    __graft_entry__._load_builder().build()
    import exact_dimensional_distance_gb300 as edd
    return edd


def test_tensor_layout_and_constants_match_header(tmp_path):
    edd = _edd()
    if shutil.which("gcc") is None:
        pytest.skip("needs gcc")
    fields = {"in": "in_", "out": "out", "n": "n", "dtype": "dtype", "reserved": "reserved"}
    src = tmp_path / "layout.c"
    src.write_text("\n".join(
        ['#include <stdio.h>', '#include <stddef.h>', '#include "hiss.h"', "int main(void) {",
         'printf("%zu %d %d %d %d %lld\\n", sizeof(hiss_tensor), HISS_F32, HISS_F16, HISS_BF16, HISS_MAX_WIDTH, '
         '(long long)HISS_NO_PAD);'] +
        ['printf("%%zu\\n", offsetof(hiss_tensor, %s));' % f for f in fields] + ["return 0; }"]))
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-I" + os.path.join(ROOT, "include"), "-o", str(exe), str(src)])
    first, *offsets = subprocess.check_output([str(exe)], text=True).splitlines()
    assert first.split() == [str(v) for v in (ctypes.sizeof(edd.hiss_tensor), edd.HISS_F32, edd.HISS_F16, edd.HISS_BF16,
                                              edd.HISS_MAX_WIDTH, edd.HISS_NO_PAD)]
    assert [int(v) for v in offsets] == [getattr(edd.hiss_tensor, f).offset for f in fields.values()]


def test_calls_without_a_context_are_refused():
    edd = _edd()
    z = edd.HISS_NO_PAD
    assert edd.hiss_embed(None, None, 0, 1, 1, 1, None, 64, 0, z, 1.0, None, 0, 1) == edd.HISS_E_ARG
    assert edd.hiss_embed_grad(None, None, 0, 1, None, 64, 0, z, 1.0, 1, 1, 0, None, 0, 1) == edd.HISS_E_ARG
    assert edd.hiss_layer_norm(None, None, 0, 1, 0, 1, None, None, 0, 1e-5, None, 0, 1, None, None) == edd.HISS_E_ARG
    assert edd.hiss_layer_norm_grad(None, None, 0, 1, None, 0, 1, None, None, None, 0, 0, 1, None, 1, None,
                                    None) == edd.HISS_E_ARG
    assert edd.hiss_clip_grads(None, None, 0, 1.0, None) == edd.HISS_E_ARG
    assert edd.hiss_finish(None) == edd.HISS_E_ARG


def test_rows_and_density():
    torch = pytest.importorskip("torch")
    edd = _edd()
    x = torch.zeros((4, 6, 8))
    m, n, d, stride = edd._matrix(x, "x")
    assert (n, d, stride, m.data_ptr()) == (24, 8, 8, x.data_ptr())
    m, n, d, stride = edd._matrix(x[0, :, :5], "x")  # a row stride of its own: no copy
    assert (n, d, stride, m.data_ptr()) == (6, 5, 8, x.data_ptr())
    m, n, d, stride = edd._matrix(x[0].t(), "x")     # columns apart: copied
    assert (n, d, stride) == (8, 6, 6) and m.data_ptr() != x.data_ptr()
    assert edd._matrix(x[0, :1].expand(9, 8), "x")[1:] == (9, 8, 0)
    for bad in (torch.zeros(()), torch.zeros((3, 0)), torch.zeros((1, edd.HISS_MAX_WIDTH + 1))):
        with pytest.raises(ValueError):
            edd._matrix(bad, "x")
    with pytest.raises(ValueError):
        edd._out_matrix(x.permute(1, 0, 2), "out")
    with pytest.raises(ValueError):
        edd._dtype(torch.float64)
    dense = edd.Gradients._dense
    assert dense(x) and dense(x.permute(2, 0, 1)) and dense(torch.zeros(())) and dense(torch.zeros((0, 3)))
    assert dense(x[:1]) and not dense(x[:, :3]) and not dense(x[0, :1].expand(5, 8)) and not dense(x[..., ::2])


def test_padding_tokens_fit_64_bits():
    edd = _edd()
    assert edd._pad(None) == edd.HISS_NO_PAD
    for pad in (0, -1, 1 << 40, (1 << 63) - 1, -(1 << 63)):
        assert edd._pad(pad) == pad
    for pad in (1 << 63, (1 << 64) - 1, -(1 << 63) - 1):  # c_int64 takes the second for -1
        with pytest.raises(ValueError):
            edd._pad(pad)
