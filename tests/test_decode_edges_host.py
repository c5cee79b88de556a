"""Host-side tests (no GPU) of what nexus_append, nexus_quantize and nexus_attend refuse and ask
for, beside those of test_decode_host.py."""
import ctypes

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
