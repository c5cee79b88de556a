"""Host-side tests (no GPU) of nexus_plan, nexus_verify and nexus_attend_shared: every refusal comes
before any CUDA call, and the tests' own plain forms hold by hand-made cases."""
import ctypes
import math
import os
import shutil

import numpy as np
import pytest
import torch

import batch_harness as H
from test_abi_host import _structs
from test_decode_host import STATUS, _image, _tok


@pytest.fixture(scope="module")
def lib():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from streaming_kv_cache_step_gb300 import build, nexus
    build.build()
    return nexus.load()


PAGED = dict(page_size=16, num_pages=1100, max_pages_per_seq=512, block_table=0x70000)


def _plan(lib, cache=None, pool="default", image=None, status=STATUS, pool_over=None, **over):
    from streaming_kv_cache_step_gb300 import nexus
    c, _ = _structs(**({**PAGED, **(cache or {})}))
    a = dict(new_tokens=0x100000, first_pos=0x110000, cu_tokens=0x120000, token_seq=0x130000,
             token_pos=0x140000, tokens=64, max_tokens=8)
    a.update(over)
    p = dict(block_table=0x70000, free_pages=0x200000, free_count=0x210000, held=0x220000,
             free_count_in=None, held_in=None)
    p.update(pool_over or {})
    pl = nexus.CPlan(*[a[n] for n, _ in nexus.CPlan._fields_])
    po = nexus.CPool(*[p[n] for n, _ in nexus.CPool._fields_])
    return lib.nexus_plan(ctypes.byref(c), ctypes.byref(po) if pool else None, ctypes.byref(pl),
                          None if image is None else ctypes.byref(image), status, None)


@pytest.mark.parametrize("bad", [
    dict(cache=dict(head_dim=96)), dict(status=None), dict(new_tokens=None), dict(cu_tokens=None),
    dict(tokens=-1), dict(max_tokens=0), dict(first_pos=None), dict(token_pos=None),
    dict(new_tokens=0x100002), dict(cu_tokens=0x120001), dict(token_seq=0x130002),
    dict(pool=None), dict(pool_over=dict(free_pages=None)), dict(pool_over=dict(free_count=None)),
    dict(pool_over=dict(held=None)), dict(pool_over=dict(block_table=0x80000)),
    dict(pool_over=dict(held_in=0x220004)), dict(pool_over=dict(free_count_in=0x210002)),
    dict(status=ctypes.c_void_p(0x900001)), dict(image="bad"),
    dict(cache=dict(page_size=0, num_pages=0, max_pages_per_seq=0, block_table=None))])
def test_plan_refuses(lib, bad):
    from streaming_kv_cache_step_gb300 import nexus
    if bad.get("image") == "bad":
        bad = dict(image=_image(rows=None))
    assert _plan(lib, **bad) == nexus.NX_ERR_INVALID_ARG


def test_plan_refuses_what_it_does_not_cover(lib):
    from streaming_kv_cache_step_gb300 import nexus
    assert _plan(lib, cache=dict(seqs=8193)) == nexus.NX_ERR_UNSUPPORTED
    assert _plan(lib, cache=dict(layers=1 << 14, kv_heads=(1 << 10) + 1, seqs=1)) == \
        nexus.NX_ERR_UNSUPPORTED
    assert _plan(lib, cache=dict(dtype=nexus.DTYPE_F32), image=_image()) == nexus.NX_ERR_UNSUPPORTED


def _verify(lib, cache=None, tok=None, image=None, status=STATUS, **over):
    from streaming_kv_cache_step_gb300 import nexus
    c, _ = _structs(**(cache or {}))
    a = dict(token=0x100000, p=0x200000, q=0x300000, p_stride=1000, q_stride=1000, u=0x400000,
             u_draw=0x410000, out=0x420000, emitted=0x430000, lens_in=None, vocab=1000,
             dtype=nexus.DTYPE_F32, reserved=0)
    a.update(over)
    st = nexus.CVerify(*[a[n] for n, _ in nexus.CVerify._fields_])
    return lib.nexus_verify(ctypes.byref(c), ctypes.byref(_tok(**(tok or {}))), ctypes.byref(st),
                            None if image is None else ctypes.byref(image), status, None)


@pytest.mark.parametrize("bad", [
    dict(cache=dict(kv_heads=0)), dict(tok=dict(tokens=3)), dict(tok=dict(max_tokens=0)),
    dict(status=None), dict(dtype=2), dict(reserved=1), dict(vocab=0), dict(p=None),
    dict(p=0x200002), dict(q=0x300001), dict(token=None), dict(u=None), dict(u_draw=None),
    dict(out=None), dict(emitted=None), dict(p_stride=-1), dict(q_stride=-4), dict(u=0x400002),
    dict(lens_in=0x40004), dict(lens_in=0x40002), dict(image="bad"), dict(out=0x100000),
    dict(out=0x100004), dict(out=0xFFFFC)])
def test_verify_refuses(lib, bad):
    from streaming_kv_cache_step_gb300 import nexus
    if bad.get("image") == "bad":
        bad = dict(image=_image(k=0x8))
    assert _verify(lib, **bad) == nexus.NX_ERR_INVALID_ARG


def test_verify_refuses_what_it_does_not_cover(lib):
    from streaming_kv_cache_step_gb300 import nexus
    assert _verify(lib, vocab=(1 << 20) + 1) == nexus.NX_ERR_UNSUPPORTED
    assert _verify(lib, cache=dict(dtype=nexus.DTYPE_F32), image=_image()) == \
        nexus.NX_ERR_UNSUPPORTED
    assert _verify(lib, dtype=nexus.DTYPE_BF16, p=0x200001) == nexus.NX_ERR_INVALID_ARG


def test_attend_shared_refuses(lib):
    from streaming_kv_cache_step_gb300 import nexus
    ws, big = ctypes.c_void_p(0x1000000), ctypes.c_size_t(1 << 40)

    def call(cache=None, pre=None, tok=None, image=None, pre_image=None, no_prefix=False,
             no_shared=False, ws=ws, size=big, status=STATUS, shared=None, bytes_only=False,
             **over):
        a = dict(q=0x100000, out=0x200000, lse=None, q_stride=4096, out_stride=4096, scale=0.1,
                 causal=1)
        a.update(over)
        c, _ = _structs(**(cache or {}))
        p, _ = _structs(**{**dict(seqs=1, k=0x50000, v=0x60000), **(pre or {})})
        x = dict(prefix=None if no_prefix else ctypes.addressof(p),
                 image=None if pre_image is None else ctypes.addressof(pre_image), cu_seqs=None,
                 max_tokens=2, reserved=0)
        x.update(shared or {})
        xs = nexus.CShared(*[x[n] for n, _ in nexus.CShared._fields_])
        st = nexus.CAttend(*[a[n] for n, _ in nexus.CAttend._fields_])
        t = _tok(**(tok or {}))
        if bytes_only:
            return lib.nexus_attend_shared_workspace_bytes(ctypes.byref(c), ctypes.byref(t),
                                                           ctypes.byref(xs))
        return lib.nexus_attend_shared(ctypes.byref(c), ctypes.byref(t),
                                       None if image is None else ctypes.byref(image),
                                       None if no_shared else ctypes.byref(xs), ctypes.byref(st),
                                       ws, size, status, None)

    of_either = (dict(cache=dict(kv_heads=0)), dict(tok=dict(layer=1)), dict(tok=dict(tokens=5)),
                 dict(no_prefix=True), dict(pre=dict(head_dim=64)), dict(pre=dict(kv_heads=4)),
                 dict(pre=dict(group=2)), dict(pre=dict(dtype=nexus.DTYPE_F32)),
                 dict(pre=dict(seqs=2)), dict(pre=dict(capacity=0)), dict(shared=dict(max_tokens=0)),
                 dict(shared=dict(reserved=1)), dict(shared=dict(cu_seqs=0x800002)),
                 dict(cache=dict(layers=2), tok=dict(layer=1)))
    for bad in of_either:
        assert call(**bad) == nexus.NX_ERR_INVALID_ARG, bad
        assert call(**bad, bytes_only=True) == 0, bad
    for bad in (dict(status=None), dict(no_shared=True), dict(q=None), dict(out=0x200004),
                dict(q_stride=4100), dict(out_stride=2048), dict(scale=math.nan),
                dict(image=_image(k=None)), dict(pre_image=_image(v=0x8)),
                dict(pre=dict(lens=0x40002))):
        assert call(**bad) == nexus.NX_ERR_INVALID_ARG, bad
    f32 = dict(cache=dict(dtype=nexus.DTYPE_F32), pre=dict(dtype=nexus.DTYPE_F32))
    assert call(**f32, image=_image()) == nexus.NX_ERR_UNSUPPORTED
    assert call(**f32, pre_image=_image()) == nexus.NX_ERR_UNSUPPORTED
    need = call(bytes_only=True)
    assert need >= 2 * 32 * (128 * 4 + 8)
    for bad in (dict(ws=None), dict(ws=ctypes.c_void_p(0x1000010)),
                dict(size=ctypes.c_size_t(need - 1))):
        assert call(**bad) == nexus.NX_ERR_WORKSPACE, bad


def test_binding_refuses_shapes_and_types():
    from streaming_kv_cache_step_gb300 import nexus
    t = torch.zeros(1, 1, 1, 64, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, 1, 1, 64, dtype=torch.int32)
    cache = nexus.Cache(k=t, v=t, pos=i, lens=i[..., 0].contiguous(), layers=1, seqs=1, kv_heads=1,
                        group=1, head_dim=64, capacity=64)
    one, two = torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    f = torch.zeros(1)
    with pytest.raises(ValueError):                                  # CPU tensors
        nexus.plan(cache, None, one, two, None, max_tokens=1, tokens=1)
    with pytest.raises(ValueError):
        nexus.verify(cache, one, torch.zeros(1, 8), f, f, one, one, None, max_tokens=1)
    with pytest.raises(ValueError):
        nexus.alloc_attend_shared_workspace(cache, cache, tokens=1, max_tokens=1, max_shared=1)


def test_binding_refuses_caches_that_do_not_fit_together(monkeypatch):
    # what would be read or written behind an array: keys and values of two types, or of one that is
    # taken for another, and too few lengths
    from streaming_kv_cache_step_gb300 import nexus

    def cache(k=torch.bfloat16, v=torch.bfloat16, lens=(2, 3, 1)):
        return nexus.Cache(k=torch.zeros(2, 3, 1, 32, 64, dtype=k), v=torch.zeros(2, 3, 1, 32, 64, dtype=v),
                           pos=torch.zeros(2, 3, 1, 32, dtype=torch.int32),
                           lens=torch.zeros(lens, dtype=torch.int32), layers=2, seqs=3, kv_heads=1,
                           group=1, head_dim=64, capacity=32)

    monkeypatch.setattr(torch.Tensor, "is_cuda", True)               # (no call gets as far as the data)
    for way in (nexus.Cache.c_struct, lambda c: nexus._packed_cache(c, -1)):
        way(cache())
        way(cache(k=torch.float32, v=torch.float32))
        for bad in (dict(v=torch.float32), dict(k=torch.float32), dict(lens=(2, 2, 1)),
                    dict(lens=(3, 3, 1)), dict(k=torch.float16, v=torch.float16)):
            with pytest.raises(ValueError):
                way(cache(**bad))


def test_packed_structures_have_the_layout_of_the_header():
    from streaming_kv_cache_step_gb300 import nexus
    for packed, c in ((nexus._CACHE, nexus.CCache), (nexus._TOKENS, nexus.CTokens),
                      (nexus._POOL, nexus.CPool), (nexus._PLAN, nexus.CPlan),
                      (nexus._VERIFY, nexus.CVerify), (nexus._ATTEND, nexus.CAttend),
                      (nexus._SHARED, nexus.CShared), (nexus._IMAGE, nexus.CImage)):
        assert packed.size == ctypes.sizeof(c)
        values = list(range(1, 1 + len(c._fields_)))
        x = c.from_buffer_copy(packed.pack(*values))
        assert [getattr(x, n) for n, _ in c._fields_] == values


def test_plain_plan_by_hand():
    # pages of 8: a grows by a page, b gives two back, c ends, d has to wait
    lens = np.zeros((2, 4, 1), np.int64)
    lens[0, :, 0] = [8, 3, 20, 9]
    lens[1, :, 0] = [7, 4, 1, 16]
    table = np.arange(40).reshape(4, 10)
    held, free = np.array([1, 3, 3, 2]), np.zeros(40, np.int64)
    cu, seq, pos, left, status = H.plan_plain(
        lens, [1, 2, -1, 60], 80, tokens=100, max_tokens=64, page=8, num_pages=40, table=table,
        free=free, count=0, held=held, first_pos=[100, 50, 0, 0])
    assert (cu, seq, pos) == ([0, 1, 3, 3, 3], [0, 1, 1], [100, 50, 51])
    assert list(free[:5]) == [11, 12, 20, 21, 22] and left == 4 and status == H.NO_PAGES
    assert list(held) == [2, 1, 0, 2] and table[0, 1] == 22
    assert lens[:, 2].max() == 0 and lens[0, 3, 0] == 9


def test_plain_verify_by_hand():
    p = np.array([[0.5, 0.5, 0, 0], [0.25, 0.25, 0.25, 0.25], [0, 0, 0, 1]], np.float32)
    q = np.array([[0, 1, 0, 0], [1, 0, 0, 0], [9, 9, 9, 9]], np.float32)
    # draft 1 stays (0.4 < 0.5), draft 0 goes (0.25 is not below 0.25), columns 1 .. 3 remain
    got = H.verify_plain([7, 1, 0], p, q, np.float32([0.4, 0.25, 0]), np.float32([0.34]), [0, 3])
    assert got == ([1, 2, -1], [2], [1], 0)
    # without q: the draft's own column goes
    got = H.verify_plain([7, 1, 0], p, None, np.float32([0.4, 0.25, 0]), np.float32([0.0]), [0, 3])
    assert got == ([1, 1, -1], [2], [1], 0)
    assert H.draw_plain(np.float32([0, 0.5, 0, 0.5]), np.float32(0.5)) == 3
    assert H.draw_plain(np.float32([0, 0.5, 0, 0.5]), np.float32(1 - 2.0 ** -24)) == 3
    assert H.draw_plain(np.float32([0, 0]), np.float32(0.1)) == -1
