"""Host-side tests (no GPU) of what nexus_append, nexus_quantize and nexus_attend refuse and ask
for, beside those of test_decode_host.py."""
import ctypes
import os
import subprocess
from types import SimpleNamespace

import pytest
import torch

from streaming_kv_cache_step_gb300 import build
from test_abi_host import _structs
from test_decode_host import STATUS, _image, _tok, lib  # noqa: F401


def test_append_image_refuses(lib):  # noqa: F811
    from streaming_kv_cache_step_gb300 import nexus

    def call(cache=None, image=None, status=STATUS, **over):
        a = dict(k=0x2000000, v=0x3000000, k_stride=1024, v_stride=1024, pos=0x5000000, eps=1e-6)
        a.update(over)
        c, _ = _structs(**(cache or {}))
        return lib.nexus_append_image(ctypes.byref(c), ctypes.byref(_tok()),
                                      ctypes.byref(nexus.CAppend(**a)),
                                      None if image is None else ctypes.byref(image), status, None)

    for bad in (dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None), dict(rows=None),
                dict(k=0x100008), dict(v=0x200001)):
        assert call(image=_image(**bad)) == nexus.NX_ERR_INVALID_ARG, bad
    for bad in (dict(status=None), dict(k_stride=1028), dict(cache=dict(head_dim=96))):
        assert call(image=_image(), **bad) == nexus.NX_ERR_INVALID_ARG, bad
        assert call(**bad) == nexus.NX_ERR_INVALID_ARG, bad
    f32 = dict(dtype=nexus.DTYPE_F32)
    assert call(cache=f32, image=_image()) == nexus.NX_ERR_UNSUPPORTED


def test_shares_of_many_tiles(tmp_path):
    # the blocks' shares follow one another without a gap up to the largest total that attend takes
    csrc = os.path.join(os.path.dirname(build.__file__), "csrc")
    src = tmp_path / "shares.cu"
    src.write_text('#include "nx_attend.cuh"\n' + "".join(
        f"""static_assert(nx::share_start({total}, nx::share_per({total}, {blocks}), 0) == 0, "");
static_assert(nx::share_start({total}, nx::share_per({total}, {blocks}), {blocks}) == {total}, "");
static_assert(nx::share_start({total}, nx::share_per({total}, {blocks}), {blocks} - 1) <= {total}, "");
static_assert(nx::share_per({total}, {blocks}) >= 1 &&
              nx::share_per({total}, {blocks}) <= {total // blocks + 1}LL, "");
""" for total in (0, 1, 455, 456, 457, 65536, 2 ** 31 - 400, 2 ** 31 - 1) for blocks in (1, 152, 304, 456)))
    p = subprocess.run([build._nvcc(), *build.ARCH, *build.FLAGS, "-I", csrc, "-c", str(src), "-o",
                        str(tmp_path / "shares.o")], capture_output=True, text=True)
    assert p.returncode == 0, p.stderr


@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("rows", [1, 16, 17, 32, 33, 80, 81, 4096])
def test_attend_workspace_goes_by_the_rows_alone(lib, rows, head_dim):  # noqa: F811
    def size(tokens, max_tokens, **cache):
        c, _ = _structs(group=1, head_dim=head_dim, **cache)
        t = _tok(tokens=tokens, max_tokens=max_tokens, cu_tokens=0x8000)
        return lib.nexus_attend_workspace_bytes(ctypes.byref(c), ctypes.byref(t))

    one = size(rows, rows, seqs=1, kv_heads=1, capacity=64)
    for cache in (dict(seqs=1, kv_heads=1, capacity=1 << 22), dict(seqs=256, kv_heads=8, capacity=512),
                  dict(seqs=64, kv_heads=8, capacity=1 << 17)):
        assert size(rows, rows, **cache) == one and size(rows, 1 << 30, **cache) == one
        assert size(1 << 20, rows, **cache) == one


class _Gpu:
    """Stands for a CUDA tensor's properties around a CPU one (no call gets as far as its data)."""

    def __init__(self, t):
        self.t, self.is_cuda = t, True

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_binding_refuses_host_memory(lib, monkeypatch):  # noqa: F811
    from streaming_kv_cache_step_gb300 import nexus
    called = lambda *a: pytest.fail("called with host memory")  # noqa: E731
    monkeypatch.setattr(nexus, "load", lambda: SimpleNamespace(
        nexus_append_image=called, nexus_quantize=called, nexus_attend=called))
    monkeypatch.setattr(nexus.Cache, "c_struct", lambda self: nexus.CCache())
    monkeypatch.setattr(nexus, "_stream", lambda stream: None)
    monkeypatch.setattr(nexus.Image, "c_struct", lambda self, cache: nexus.CImage())
    z = lambda *s, dt=torch.bfloat16: _Gpu(torch.zeros(*s, dtype=dt))  # noqa: E731
    i = lambda *s: z(*s, dt=torch.int32)  # noqa: E731
    cache = nexus.Cache(k=z(1, 1, 1, 64, 64), v=z(1, 1, 1, 64, 64), pos=i(1, 1, 1, 64), lens=i(1, 1, 1),
                        layers=1, seqs=1, kv_heads=1, group=1, head_dim=64, capacity=64)
    q, kv, pos, st, ws = z(1, 1, 64), z(1, 1, 64), i(1), i(1), z(4096, dt=torch.uint8)
    rot = nexus.Rotary([1.0] * 4, device="cpu")
    on = nexus.Rotary([1.0] * 4, device="cpu")
    on.table = _Gpu(on.table)

    def append(status=st, rotary=on):
        nexus.append(cache, 0, q, kv, kv, pos, q, status, max_tokens=1, rotary=rotary)

    def attend(status=st, ws=ws):
        nexus.attend(cache, 0, q, q, ws, status, max_tokens=1)

    host, wrong = torch.zeros(1, dtype=torch.int32), z(1, dt=torch.float32)
    for call in (lambda: append(rotary=rot), lambda: append(status=host), lambda: append(status=None),
                 lambda: append(status=wrong), lambda: attend(status=host), lambda: attend(status=wrong),
                 lambda: attend(ws=torch.zeros(4096, dtype=torch.uint8)),
                 lambda: nexus.quantize(cache, nexus.Image(*[None] * 5), host)):
        with pytest.raises(ValueError):
            call()


def test_misaligned_counts_and_scales_are_refused(lib):  # noqa: F811
    from streaming_kv_cache_step_gb300 import nexus
    big = ctypes.c_size_t(1 << 40)

    def append(cache=None, tok=None, status=STATUS, **over):
        a = dict(k=0x2000000, v=0x3000000, k_stride=1024, v_stride=1024, pos=0x5000000, eps=1e-6)
        c, _ = _structs(**(cache or {}))
        return lib.nexus_append(ctypes.byref(c), ctypes.byref(_tok(**(tok or {}))),
                                ctypes.byref(nexus.CAppend(**{**a, **over})), status, None)

    def attend(cache=None, tok=None, image=None, status=STATUS, **over):
        a = dict(q=0x100000, out=0x200000, q_stride=4096, out_stride=4096, scale=0.1, causal=1)
        c, _ = _structs(**(cache or {}))
        return lib.nexus_attend(ctypes.byref(c), ctypes.byref(_tok(**(tok or {}))),
                                None if image is None else ctypes.byref(image),
                                ctypes.byref(nexus.CAttend(**{**a, **over})),
                                ctypes.c_void_p(0x1000000), big, status, None)

    def quantize(cache=None, rows_in=None, status=STATUS, **im):
        c, _ = _structs(**(cache or {}))
        return lib.nexus_quantize(ctypes.byref(c), ctypes.byref(_image(**im)), rows_in, status, None)

    off = ctypes.c_void_p(0x900002)
    cu = dict(tok=dict(cu_tokens=0x8001))
    for call in (lambda: append(pos=0x5000002), lambda: append(lens_in=0x7000001),
                 lambda: append(status=off), lambda: append(**cu),
                 lambda: append(cache=dict(lens=0x40002)), lambda: append(cache=dict(pos=0x30001)),
                 lambda: attend(lse=0x300002), lambda: attend(status=off), lambda: attend(**cu),
                 lambda: attend(cache=dict(lens=0x40001)),
                 lambda: attend(image=_image(rows=0x500002)),
                 lambda: attend(image=_image(k_scale=0x300001)),
                 lambda: quantize(rows_in=ctypes.c_void_p(0x600003)), lambda: quantize(status=off),
                 lambda: quantize(v_scale=0x400002), lambda: quantize(cache=dict(lens=0x40002))):
        assert call() == nexus.NX_ERR_INVALID_ARG


def test_attend_refuses_more_rows_than_it_counts(lib):  # noqa: F811
    from streaming_kv_cache_step_gb300 import nexus

    def call(tokens):
        c, _ = _structs(seqs=1, kv_heads=1, group=1 << 20, head_dim=64, capacity=64)
        a = nexus.CAttend(q=0x100000, out=0x200000, q_stride=1 << 26, out_stride=1 << 26, scale=0.1, causal=1)
        return lib.nexus_attend(ctypes.byref(c), ctypes.byref(_tok(tokens=tokens, max_tokens=tokens)), None,
                                ctypes.byref(a), ctypes.c_void_p(0x1000000), ctypes.c_size_t(0), STATUS, None)

    assert call(2048) == nexus.NX_ERR_UNSUPPORTED
    assert call(2047) == nexus.NX_ERR_WORKSPACE                      # taken, but for the workspace
