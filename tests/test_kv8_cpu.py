"""CPU-side checks of the 8-bit K/V cache's boundary: struct layouts, the argument checks of
the library before any CUDA call, and the binding's refusals."""
import ctypes
import os
import subprocess
import tempfile
import types

import pytest
import torch

import flow_matching_vla_euler_b200 as V
from flow_matching_vla_euler_b200 import build as B


@pytest.fixture(scope="module")
def lib():
    B.build()
    return V.load_library()


def test_struct_layout_matches_header():
    src = r"""
    #include <stdio.h>
    #include <stddef.h>
    #include "vla.h"
    int main(void) {
      printf("%zu %zu %zu %zu %zu %zu %zu %zu %zu\n", sizeof(vla_kv8_config), offsetof(vla_kv8_config, flags),
             sizeof(vla_kv8_rows), offsetof(vla_kv8_rows, layer), offsetof(vla_kv8_rows, stride),
             sizeof(vla_kv8_query), offsetof(vla_kv8_query, layer), offsetof(vla_kv8_query, scale),
             offsetof(vla_kv8_query, out_stride));
      return 0;
    }
    """
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        with open(c, "w") as f:
            f.write(src)
        subprocess.check_call(["gcc", "-I", os.path.dirname(V.HEADER_PATH), c, "-o", exe])
        got = [int(x) for x in subprocess.check_output([exe]).decode().split()]
    assert got == [ctypes.sizeof(V.vla_kv8_config), V.vla_kv8_config.flags.offset, ctypes.sizeof(V.vla_kv8_rows),
                   V.vla_kv8_rows.layer.offset, V.vla_kv8_rows.stride.offset, ctypes.sizeof(V.vla_kv8_query),
                   V.vla_kv8_query.layer.offset, V.vla_kv8_query.scale.offset, V.vla_kv8_query.out_stride.offset]


def test_create_and_null_arguments(lib):
    h = ctypes.c_void_p()

    def cfg(**kw):
        c = V.vla_kv8_config()
        for k, v in dict(dict(n_layers=1, n_kv_heads=1, head_dim=64, capacity=64, n_slots=1, flags=0), **kw).items():
            setattr(c, k, v)
        return c

    assert lib.vla_kv8_create(None, ctypes.byref(h)) == V.VLA_ERR_ARG
    assert lib.vla_kv8_create(ctypes.byref(cfg()), None) == V.VLA_ERR_ARG
    assert lib.vla_kv8_create(ctypes.byref(cfg(flags=1)), ctypes.byref(h)) == V.VLA_ERR_ARG
    for bad in [dict(n_layers=0), dict(n_kv_heads=0), dict(capacity=0), dict(n_slots=0), dict(head_dim=48),
                dict(head_dim=512), dict(capacity=-1), dict(capacity=(1 << 30) + 1),
                dict(n_layers=64, n_kv_heads=64, head_dim=256, capacity=1 << 20, n_slots=64)]:
        assert lib.vla_kv8_create(ctypes.byref(cfg(**bad)), ctypes.byref(h)) == V.VLA_ERR_SHAPE, bad
        assert not h.value
    rows, args = V.vla_kv8_rows(), V.vla_kv8_query()
    one = ctypes.c_void_p(256)
    assert lib.vla_kv8_write(None, one, one, ctypes.byref(rows), None) == V.VLA_ERR_ARG
    assert lib.vla_kv8_read(None, one, one, ctypes.byref(rows), None) == V.VLA_ERR_ARG
    assert lib.vla_kv8_attend(None, one, one, None, ctypes.byref(args), None) == V.VLA_ERR_ARG
    assert lib.vla_kv8_status(None, None) == V.VLA_ERR_ARG
    lib.vla_kv8_destroy(None)


def _cache():
    return types.SimpleNamespace(n_layers=2, n_kv_heads=2, head_dim=32, capacity=100, n_slots=3, device=0, handle=None,
                                 _here=V.KVCache8._here, _index=V.KVCache8._index, _strided=V.KVCache8._strided)


def test_binding_shapes():
    c = _cache()
    for name in ("_here", "_index", "_strided"):
        setattr(c, name, types.MethodType(getattr(V.KVCache8, name), c))
    k = torch.zeros(2, 3, 5, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="K"):
        V.KVCache8.write(c, k[0], k[0])
    with pytest.raises(ValueError, match="K"):
        V.KVCache8.write(c, k[..., :32], k)
    with pytest.raises(ValueError, match="go together"):
        V.KVCache8.read(c, 5, K_out=k)
    with pytest.raises(ValueError, match="K_out"):
        V.KVCache8.read(c, 4, K_out=k, V_out=k)
    with pytest.raises(ValueError, match="q"):
        V.KVCache8.attend(c, k[0], torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="q"):
        V.KVCache8.attend(c, k, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="scale"):
        V.KVCache8.attend(c, torch.zeros(2, 1, 4, 32, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32), scale=0.0)
    # host tensors of the right shape reach the check for CUDA
    with pytest.raises(TypeError, match="CUDA"):
        V.KVCache8.write(c, k, k)
    with pytest.raises(TypeError, match="CUDA"):
        V.KVCache8.attend(c, torch.zeros(2, 1, 4, 32, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32))


@pytest.mark.parametrize("scale", [1e-50, 7e-46, -1.0, 0.0, float("nan")])
def test_scales_that_fp32_does_not_hold(scale):
    """A scale that fp32 makes 0 would reach the library as the default."""
    c = _cache()
    q = torch.zeros(2, 1, 4, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="scale"):
        V.KVCache8.attend(c, q, torch.zeros(2, dtype=torch.int32), scale=scale)


def test_create_without_a_gpu_fails_cleanly(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    with pytest.raises(V.VlaError) as ei:
        V.KVCache8(n_layers=1, n_kv_heads=1, head_dim=64, capacity=64)
    assert ei.value.code in (V.VLA_ERR_CUDA, V.VLA_ERR_UNSUPPORTED)
