"""Host-side tests (no GPU) of nexus_append, nexus_quantize and nexus_attend: every refusal
comes before any CUDA call, and the binding's own checks and tables hold."""
import ctypes
import math
import os
import shutil
from fractions import Fraction

import numpy as np
import pytest
import torch

from decode_harness import e4m3_grid, quantize64
from test_abi_host import _structs


@pytest.fixture(scope="module")
def lib():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from streaming_kv_cache_step_gb300 import build, nexus
    build.build()
    return nexus.load()


def _tok(**over):
    from streaming_kv_cache_step_gb300 import nexus
    t = dict(layer=0, tokens=2, max_tokens=1, reserved=0, cu_tokens=None)
    t.update(over)
    return nexus.CTokens(*[t[n] for n, _ in nexus.CTokens._fields_])


STATUS = ctypes.c_void_p(0x900000)


def _append(lib, cache=None, tok=None, status=STATUS, **over):
    from streaming_kv_cache_step_gb300 import nexus
    a = dict(q=0x1000000, k=0x2000000, v=0x3000000, q_stride=4096, k_stride=1024, v_stride=1024,
             q_out=0x4000000, pos=0x5000000, lens_in=None, rotary=0x6000000, rotary_dim=128,
             interleaved=0, q_norm=None, k_norm=None, eps=1e-6, reserved=0)
    a.update(over)
    c, _ = _structs(**(cache or {}))
    st = nexus.CAppend(*[a[n] for n, _ in nexus.CAppend._fields_])
    return lib.nexus_append(ctypes.byref(c), ctypes.byref(_tok(**(tok or {}))), ctypes.byref(st),
                            status, None)


@pytest.mark.parametrize("bad", [
    dict(cache=dict(head_dim=96)), dict(cache=dict(dtype=3)), dict(cache=dict(k=0x10008)),
    dict(tok=dict(layer=1)), dict(tok=dict(layer=-1)), dict(tok=dict(tokens=3)),
    dict(tok=dict(tokens=-1)), dict(tok=dict(max_tokens=0)), dict(tok=dict(reserved=1)),
    dict(status=None), dict(reserved=1), dict(eps=-1.0), dict(eps=math.inf), dict(eps=math.nan),
    dict(rotary_dim=12), dict(rotary_dim=136), dict(rotary_dim=-8), dict(rotary_dim=0),
    dict(rotary=None), dict(rotary=0x6000004), dict(q=None), dict(q_out=None), dict(k=None),
    dict(v=None), dict(pos=None), dict(k=0x2000008), dict(q=0x1000002), dict(q_out=0x4000008),
    dict(k_stride=1028), dict(v_stride=-1024), dict(q_stride=4097), dict(q_norm=0x7000008),
    dict(k_norm=0x7000002), dict(q_out=0x1000000, q_stride=8192), dict(lens_in=0x40004)])
def test_append_refuses(lib, bad):
    from streaming_kv_cache_step_gb300 import nexus
    assert _append(lib, **bad) == nexus.NX_ERR_INVALID_ARG


def test_append_refuses_too_many_heads(lib):
    from streaming_kv_cache_step_gb300 import nexus
    assert _append(lib, cache=dict(kv_heads=8193)) == nexus.NX_ERR_UNSUPPORTED


def _image(**over):
    from streaming_kv_cache_step_gb300 import nexus
    i = dict(k=0x100000, v=0x200000, k_scale=0x300000, v_scale=0x400000, rows=0x500000)
    i.update(over)
    return nexus.CImage(*[i[n] for n, _ in nexus.CImage._fields_])


def test_quantize_refuses(lib):
    from streaming_kv_cache_step_gb300 import nexus

    def call(cache=None, rows_in=None, status=STATUS, **im):
        c, _ = _structs(**(cache or {}))
        return lib.nexus_quantize(ctypes.byref(c), ctypes.byref(_image(**im)), rows_in, status, None)

    for bad in (dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None),
                dict(rows=None), dict(k=0x100008), dict(v=0x200001), dict(status=None),
                dict(cache=dict(capacity=0)), dict(rows_in=ctypes.c_void_p(0x500004))):
        assert call(**bad) == nexus.NX_ERR_INVALID_ARG, bad
    assert call(cache=dict(dtype=nexus.DTYPE_F32)) == nexus.NX_ERR_UNSUPPORTED


def test_attend_refuses(lib):
    from streaming_kv_cache_step_gb300 import nexus
    ws, big = ctypes.c_void_p(0x1000000), ctypes.c_size_t(1 << 40)

    def call(cache=None, tok=None, image=None, ws=ws, size=big, status=STATUS, **over):
        a = dict(q=0x100000, out=0x200000, lse=None, q_stride=4096, out_stride=4096, scale=0.1,
                 causal=1)
        a.update(over)
        c, _ = _structs(**(cache or {}))
        st = nexus.CAttend(*[a[n] for n, _ in nexus.CAttend._fields_])
        return lib.nexus_attend(ctypes.byref(c), ctypes.byref(_tok(**(tok or {}))),
                                None if image is None else ctypes.byref(image), ctypes.byref(st),
                                ws, size, status, None)

    for bad in (dict(cache=dict(kv_heads=0)), dict(tok=dict(layer=2)), dict(tok=dict(tokens=5)),
                dict(status=None), dict(q=None), dict(out=None), dict(q=0x100008),
                dict(out=0x200004), dict(q_stride=4100), dict(out_stride=2048),
                dict(out_stride=-4096), dict(scale=math.nan), dict(scale=math.inf),
                dict(image=_image(k=None)), dict(image=_image(v=0x8))):
        assert call(**bad) == nexus.NX_ERR_INVALID_ARG, bad
    assert call(cache=dict(dtype=nexus.DTYPE_F32), image=_image()) == nexus.NX_ERR_UNSUPPORTED
    for bad in (dict(ws=None), dict(ws=ctypes.c_void_p(0x1000010)), dict(size=ctypes.c_size_t(16))):
        assert call(**bad) == nexus.NX_ERR_WORKSPACE, bad


def test_attend_workspace_bytes(lib):
    c, _ = _structs()
    assert lib.nexus_attend_workspace_bytes(ctypes.byref(c), ctypes.byref(_tok())) >= 256
    for bad in (dict(layer=-1), dict(tokens=7), dict(max_tokens=0), dict(reserved=2)):
        assert lib.nexus_attend_workspace_bytes(ctypes.byref(c), ctypes.byref(_tok(**bad))) == 0
    c, _ = _structs(head_dim=80)
    assert lib.nexus_attend_workspace_bytes(ctypes.byref(c), ctypes.byref(_tok())) == 0


def test_rotary_table_is_the_frequency_in_turns():
    from streaming_kv_cache_step_gb300 import nexus
    freqs = [1.0, 0.1, -0.25, 1e-7, 7.5, 2.0 ** -40, 0.0, 500000.0 ** -0.5]
    r = nexus.Rotary(freqs, device="cpu")
    assert r.rotary_dim == 16 and r.table.dtype == torch.int64
    for f, t in zip(freqs, r.table.tolist()):
        for p in (1, 12345, (1 << 31) - 1, -3):
            turn = Fraction((p * t) % (1 << 64), 1 << 64)        # as the kernel multiplies
            ang = 2 * math.pi * float(turn)
            err = max(abs(math.cos(ang) - math.cos(math.fmod(p * f, 2 * math.pi))),
                      abs(math.sin(ang) - math.sin(math.fmod(p * f, 2 * math.pi))))
            # the reference's product and remainder err by ulps of the angle, 2^-53 |p f|
            assert err <= 2.0 ** -51 * abs(p * f) + 1e-9 * (abs(p) / 2.0 ** 31) + 1e-15
    for bad in ([], [1.0], [1.0] * 5, [1.0, 2.0, math.nan, 3.0], [math.inf] * 4):
        with pytest.raises(ValueError):
            nexus.Rotary(bad, device="cpu")


def test_binding_refuses_shapes_and_types():
    from streaming_kv_cache_step_gb300 import nexus
    t = torch.zeros(1, 1, 1, 64, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, 1, 1, 64, dtype=torch.int32)
    cache = nexus.Cache(k=t, v=t, pos=i, lens=i[..., 0].contiguous(), layers=1, seqs=1, kv_heads=1,
                        group=1, head_dim=64, capacity=64)
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):                                  # CPU tensors
        nexus.append(cache, 0, q, q, q, torch.zeros(1, dtype=torch.int32), q, None, max_tokens=1)
    with pytest.raises(ValueError):
        nexus.attend(cache, 0, q, q, q, None, max_tokens=1)
    im = nexus.new_image(cache)
    assert im.k.shape == t.shape and im.k_scale.shape == (1, 1, 1, 2)
    with pytest.raises(ValueError):
        im.c_struct(cache)


def test_plain_quantiser_rounds_to_the_grid():
    # the tests' own quantiser against torch's conversion, values within range
    x = torch.randn(32, 64, generator=torch.Generator().manual_seed(1))
    val, scale = quantize64(x)
    assert x.abs().max() <= 448 * scale < 2 * x.abs().max() + 1e-30
    ref = (x / scale).to(torch.float8_e4m3fn).double()
    assert np.array_equal(val, ref.numpy())
    assert len(e4m3_grid()) == 127 and e4m3_grid().max() == 448
