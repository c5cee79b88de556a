"""nexus_append, nexus_quantize and nexus_attend on the GPU against plain 64-bit forms.

Tolerances, in units of what rounds. Half a step of bf16 is 2^-8 of a value, of fp32 2^-24.
append: the result is rounded once (2^-8 or 2^-24 of it); before that, sums of at most
head_dim squares, a square root, a division and two products act in fp32, on pairs, at most
about 16 roundings: 2^-20 of the pair's magnitudes. attend: the output's rounding (2^-8 of it
for bf16), the probabilities' (2^-8 of sum p |v| / sum p for bf16 caches, 2^-11 from the
image; fp32 caches: terms of 2^-21 each, 2^-19 together) and what an error dx of the logits
changes (2 dx of the same sum): dx <= 2^-24 (d + 8) scale sum |q_i k_i| for exact products
summed in fp32, and 2^-20 scale sum |q_i k_i| for fp32 caches. lse errs by dx and two fp32
roundings of a sum of T terms (2^-19)."""
import math

import numpy as np
import pytest
import torch

from decode_harness import DEV, Case, attend64, norm64, quantize64, rotate64
from streaming_kv_cache_step_gb300 import nexus

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def _status():
    return nexus.new_status(torch.device(DEV))


def _freqs(r, theta=500000.0):
    return [theta ** (-2.0 * i / r) for i in range(r // 2)]


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

APPENDS = {
    # one token, the smallest cache
    "one": dict(case=dict(kv_heads=1, group=1, capacity=1), n=[1]),
    "decode": dict(case=dict(seqs=3, kv_heads=4, group=3, capacity=100, lens=[[5], [0], [99]]),
                   n=None, max_tokens=1, norm=True),
    "ragged": dict(case=dict(seqs=4, kv_heads=2, group=2, capacity=90, lens=[[3, 40], [0, 1], [7, 7], [31, 5]]),
                   n=[17, 0, 5, 50], norm=True, packed=True),
    "paged8": dict(case=dict(seqs=3, kv_heads=3, group=1, page=8, capacity=64, lens=[[7, 8, 9], [0, 1, 2], [30, 3, 16]]),
                   n=[9, 1, 30], rotary=64, interleaved=True),
    "paged128": dict(case=dict(seqs=2, kv_heads=2, group=4, d=64, page=128, capacity=256, lens=[[100, 127], [128, 129]]),
                     n=[64, 33], rotary=16, norm=True),
    "f32": dict(case=dict(seqs=2, kv_heads=2, group=2, d=64, dtype=F32, capacity=77, lens=[[1, 2], [3, 4]]),
                n=[3, 70], rotary=32, interleaved=True, norm=True),
    "f32_128": dict(case=dict(seqs=1, kv_heads=5, group=1, dtype=F32, page=16, capacity=48, lens=11),
                    n=[21], norm=True, packed=True),
    "no_rotary": dict(case=dict(seqs=2, kv_heads=2, group=2, capacity=33), n=[33, 2], rotary=0),
    "rotary_8": dict(case=dict(kv_heads=2, group=2, d=64, capacity=33), n=[9], rotary=8),
    "rotary_40": dict(case=dict(kv_heads=2, group=2, capacity=33), n=[9], rotary=40),
    "rotary_24_pairs": dict(case=dict(kv_heads=2, group=2, capacity=33), n=[9], rotary=24,
                            interleaved=True),
    "layer": dict(case=dict(seqs=2, layers=3, kv_heads=2, capacity=20, lens=4), n=[2, 3], layer=1),
    "kv_only": dict(case=dict(seqs=2, kv_heads=2, capacity=20, lens=4), n=[2, 3], q=False, norm=True),
    "many_heads": dict(case=dict(seqs=1, kv_heads=70, group=2, d=64, capacity=9), n=[3], norm=True),
}


def _append_inputs(c, n, packed, norm, far):
    HG, H, d, N = c.H * c.G, c.H, c.d, int(sum(n))
    x = torch.randn(N, HG + 2 * H, d, generator=c.g).to(c.dtype)
    w = [(1 + 0.3 * torch.randn(d, generator=c.g)).to(c.dtype) if norm else None
         for _ in range(2)]
    pos = torch.as_tensor(np.concatenate([far + 1000 * s + np.arange(m) for s, m in enumerate(n)])
                          .astype(np.int32)) if N else torch.zeros(0, dtype=torch.int32)
    dev = x.to(DEV)
    parts = dev[:, :HG], dev[:, HG:HG + H], dev[:, HG + H:]
    if not packed:
        parts = tuple(p.contiguous() for p in parts)
    return x, parts, w, pos


def _run_append(name, far=(1 << 30) + 12345, in_place=True):
    spec = dict(APPENDS[name])
    c = Case(**spec["case"], seed=len(name))
    n = spec["n"] if spec["n"] is not None else [spec["max_tokens"]] * c.S
    layer, r = spec.get("layer", 0), spec.get("rotary", c.d)
    inter, norm = spec.get("interleaved", False), spec.get("norm", False)
    x, (q, k, v), (wq, wk), pos = _append_inputs(c, n, spec.get("packed", False), norm, far)
    HG, H = c.H * c.G, c.H
    with_q = spec.get("q", True)
    cache, st = c.device_cache(), _status()
    rot = nexus.Rotary(_freqs(r), interleaved=inter, device=DEV) if r else None
    q_out = torch.full((len(pos), HG, c.d), math.nan, dtype=c.dtype, device=DEV)
    lens_in = None
    if not in_place:                       # the cache's own lengths are then not read
        lens_in = cache.lens[layer].clone()
        cache.lens[layer] = 12345
    put = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    nexus.append(cache, layer, q if with_q else None, k, v, put(pos), q_out if with_q else None,
                 st, max_tokens=max(max(n), 1), cu_tokens=None if spec["n"] is None else put(c.cu(n)),
                 lens_in=lens_in, rotary=rot, q_norm=put(wq) if with_q else None, k_norm=put(wk),
                 eps=1e-5)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    fr = _freqs(r) if r else []
    pre_q, pre_k = norm64(x[:, :HG], wq, 1e-5), norm64(x[:, HG:HG + H], wk, 1e-5)
    ref_q, ref_k = rotate64(pre_q, pos, fr, inter), rotate64(pre_k, pos, fr, inter)

    def close(got, ref, pre):
        row = pre.abs().amax(-1, keepdim=True)
        tol = HALF[c.dtype] * ref.abs() + 2.0 ** -20 * 2 * row + 2.0 ** -120
        err = (got.cpu().double() - ref).abs()
        assert torch.all(err <= tol), (err / tol).max()

    if with_q:
        close(q_out, ref_q, pre_q)
    want_k, want_v, want_pos = c.k.clone(), c.v.clone(), c.pos.clone()
    want_lens, a = c.lens.copy(), 0
    K, V, P = cache.k.cpu(), cache.v.cpu(), cache.pos.cpu()
    for s, m in enumerate(n):
        for h in range(H):
            old = int(c.lens[layer, s, h])
            at = c.at(layer, s, h, old + m, old)
            close(K[at], ref_k[a:a + m, h], pre_k[a:a + m, h])
            want_k[at], want_v[at], want_pos[at] = K[at], x[a:a + m, HG + H + h], pos[a:a + m]
            want_lens[layer, s, h] = old + m
        a += m
    bits = torch.int16 if c.dtype == BF else torch.int32
    assert torch.equal(K.view(bits), want_k.view(bits))      # nothing else was written
    assert torch.equal(V.view(bits), want_v.view(bits))
    assert torch.equal(P, want_pos)
    assert np.array_equal(cache.lens.cpu().numpy(), want_lens)


@pytest.mark.parametrize("in_place", [True, False], ids=["in_place", "lens_in"])
@pytest.mark.parametrize("name", list(APPENDS))
def test_append_matches_plain(name, in_place):
    _run_append(name, in_place=in_place)


@pytest.mark.parametrize("far", [0, 1, 131071, (1 << 24) + 1, (1 << 31) - 5000])
def test_append_rotates_far_positions_exactly(far):
    _run_append("f32", far=far)


def test_append_takes_drafts_back_and_queries_in_place():
    c = Case(seqs=2, kv_heads=2, group=2, capacity=32, lens=[[5, 6], [7, 8]])
    cache, st = c.device_cache(), _status()
    base = cache.lens[0].clone()
    rot = nexus.Rotary(_freqs(128), device=DEV)
    pos = torch.arange(8, dtype=torch.int32, device=DEV)
    outs = []
    for _ in range(2):                      # the second draft replaces the first
        q, k, v = (torch.randn(8, h, 128, generator=c.g).to(DEV, BF) for h in (4, 2, 2))
        ref = torch.empty_like(q)
        nexus.append(cache, 0, q, k, v, pos, ref, st, max_tokens=4, lens_in=base, rotary=rot)
        nexus.append(cache, 0, q, k, v, pos, q, st, max_tokens=4, lens_in=base, rotary=rot)
        torch.cuda.synchronize()
        assert torch.equal(q, ref)
        assert torch.equal(cache.lens[0], base + 4)
        outs.append((cache.k.clone(), v))
    a, b = outs
    assert not torch.equal(torch.nan_to_num(a[0]), torch.nan_to_num(b[0]))
    assert torch.equal(cache.v[0, 1, 0, 7:11], b[1][4:, 0])
    assert int(st.item()) == 0


def test_append_faults_are_flagged_and_leave_the_slice():
    for page in (0, 8):
        c = Case(seqs=3, kv_heads=2, group=1, page=page, capacity=16, lens=[[3, 3], [12, 3], [3, 3]])
        cache, st = c.device_cache(), _status()
        cache.lens[0, 2, 1] = 99                                     # beyond the capacity
        before = cache.lens.clone()
        q, k, v = (torch.ones(15, h, 128, dtype=BF, device=DEV) for h in (2, 2, 2))
        pos = torch.zeros(15, dtype=torch.int32, device=DEV)
        q_out = torch.zeros_like(q)
        kb = cache.k.clone()
        nexus.append(cache, 0, q, k, v, pos, q_out, st, max_tokens=5)
        torch.cuda.synchronize()
        assert int(st.item()) == nexus.NX_DEV_FULL | nexus.NX_DEV_BAD_LEN
        want = before + 5
        want[0, 1, 0], want[0, 2, 1] = 12, 99
        assert torch.equal(cache.lens, want)
        at = c.at(0, 1, 0, 16)
        assert torch.equal(cache.k.cpu()[at].view(torch.int16), kb.cpu()[at].view(torch.int16))
        # token ranges that run backwards, are too long or leave the array
        for cu, bad in (([0, 5, 3, 6], 1), ([0, 6, 7, 8], 0), ([0, 1, 2, 99], 2), ([-1, 2, 3, 4], 0)):
            st.zero_()
            cache.lens.copy_(torch.full_like(before, 2))
            nexus.append(cache, 0, q, k, v, pos, q_out, st, max_tokens=5,
                         cu_tokens=torch.tensor(cu, dtype=torch.int32, device=DEV))
            torch.cuda.synchronize()
            assert int(st.item()) == nexus.NX_DEV_BAD_TOKENS
            assert torch.all(cache.lens[0, bad] == 2)


def test_append_bad_page_is_skipped():
    c = Case(seqs=1, kv_heads=2, group=1, page=8, capacity=24, lens=6)
    cache, st = c.device_cache(), _status()
    cache.block_table[0, 1] = 1000
    x = torch.ones(5, 2, 128, dtype=BF, device=DEV)
    before = cache.k.clone()
    nexus.append(cache, 0, None, x, x, torch.zeros(5, dtype=torch.int32, device=DEV), None, st,
                 max_tokens=5)
    torch.cuda.synchronize()
    assert int(st.item()) == nexus.NX_DEV_BAD_PAGE
    before[0, int(c.table[0, 0]), :, 6:] = 1
    assert torch.equal(cache.k.view(torch.int16), before.view(torch.int16))


# ---------------------------------------------------------------------------
# quantize
# ---------------------------------------------------------------------------

QUANTS = {
    "contiguous": dict(seqs=2, kv_heads=3, layers=2, capacity=150, lens=[[0, 31, 32], [33, 64, 150]]),
    "d64": dict(seqs=1, kv_heads=2, d=64, capacity=100, lens=[[100, 63]]),
    "page8": dict(seqs=2, kv_heads=2, page=8, capacity=64, lens=[[7, 64], [8, 23]]),
    "page16_d64": dict(seqs=2, kv_heads=2, d=64, page=16, capacity=64, lens=[[15, 64], [16, 40]]),
    "page8_d64": dict(seqs=2, kv_heads=1, d=64, page=8, capacity=40, lens=[[9], [40]]),
    "page32": dict(seqs=3, kv_heads=2, page=32, capacity=96, lens=[[31, 32], [33, 96], [0, 64]]),
    "page128": dict(seqs=2, kv_heads=2, layers=2, page=128, capacity=256, lens=[[200, 129], [31, 256]]),
}


def _image(c, cache):
    im = nexus.new_image(cache)
    im.k.view(torch.uint8).fill_(0x7F)                               # NaN
    im.v.view(torch.uint8).fill_(0x7F)
    im.k_scale.fill_(math.nan)
    im.v_scale.fill_(math.nan)
    return im


def _scale_at(c, l, s, h, j):
    if c.page:
        return l, int(c.table[s, j // c.page]), h, j % c.page // c.b
    return l, s, h, j // c.b


@pytest.mark.parametrize("in_place", [True, False], ids=["in_place", "rows_in"])
@pytest.mark.parametrize("name", list(QUANTS))
def test_quantize_is_exact(name, in_place):
    c = Case(**QUANTS[name], seed=3)
    # rows of very different sizes; zeros, subnormals, ties, infinities and NaN among them
    for t in (c.k, c.v):
        t *= torch.exp2(torch.randint(-20, 20, c.shape, generator=c.g)[..., None].float()).to(BF)
    at = c.at(0, 0, c.H - 1, int(c.lens[0, 0, c.H - 1]))
    rows = c.k[at]
    if rows.shape[0] >= c.b:
        rows[:c.b] = 0
        rows[c.b:2 * c.b] *= 2.0 ** -120
        c.k[at] = rows
    at = c.at(0, c.S - 1, c.H - 1, int(c.lens[0, c.S - 1, c.H - 1]))
    rows = c.v[at]
    if rows.shape[0] >= c.b:
        rows[0, :4] = torch.tensor([math.inf, -math.inf, math.nan, -0.0])
        rows[1, :8] = torch.tensor([448., 1.0625, 1.1875, 17., 19., -17., 2. ** -10, 3 * 2. ** -10])
        c.v[at] = rows
    cache, st = c.device_cache(), _status()
    im = _image(c, cache)
    held = (torch.as_tensor(c.lens) // 2 // c.b * c.b).to(DEV)
    if in_place:
        im.rows.copy_(held)
        nexus.quantize(cache, im, st)
    else:
        im.rows.fill_(777)
        nexus.quantize(cache, im, st, rows_in=held)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert np.array_equal(im.rows.cpu().numpy(), c.lens // c.b * c.b)
    for t, q, sc in ((c.k, im.k, im.k_scale), (c.v, im.v, im.v_scale)):
        want = torch.full(c.k.shape, math.nan)
        want_s = torch.full(sc.shape, math.nan)
        for l in range(c.L):
            for s in range(c.S):
                for h in range(c.H):
                    n = int(c.lens[l, s, h])
                    for j in range(n // 2 // c.b * c.b, n // c.b * c.b, c.b):
                        at = c.at(l, s, h, j + c.b, j)
                        val, scale = quantize64(t[at])
                        want[at] = torch.as_tensor(val).float()
                        want_s[_scale_at(c, l, s, h, j)] = scale
        got = q.cpu().float()
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.nan_to_num(), want.nan_to_num())
        assert torch.equal(sc.cpu().isnan(), want_s.isnan())
        assert torch.equal(sc.cpu().nan_to_num(), want_s.nan_to_num())


def test_quantize_faults_are_flagged():
    c = Case(seqs=1, kv_heads=4, page=32, capacity=96, lens=[[64, 64, 64, 64]])
    cache, st = c.device_cache(), _status()
    im = _image(c, cache)
    im.rows.copy_(torch.tensor([[[96, 31, -32, 0]]]))
    before = im.rows.clone()
    nexus.quantize(cache, im, st)
    torch.cuda.synchronize()
    assert int(st.item()) == nexus.NX_DEV_BAD_IMAGE
    before[0, 0, 3] = 64
    assert torch.equal(im.rows, before)
    st.zero_()
    im.rows.zero_()
    cache.lens[0, 0, 3] = 97
    nexus.quantize(cache, im, st)
    torch.cuda.synchronize()
    assert int(st.item()) == nexus.NX_DEV_BAD_LEN
    st.zero_()
    cache.lens.fill_(64)
    im.rows.zero_()
    cache.block_table[0, 1] = -1
    nexus.quantize(cache, im, st)
    torch.cuda.synchronize()
    assert int(st.item()) == nexus.NX_DEV_BAD_PAGE


# ---------------------------------------------------------------------------
# attend
# ---------------------------------------------------------------------------

def _check_attend(c, n, layer=0, causal=True, image=False, scale=None, uniform=False, qscale=1.0,
                  packed_out=True, held=None, mutate=None):
    """held: rows the image holds, [layers][seqs][kv_heads] (default: all full blocks)."""
    HG, N = c.H * c.G, int(sum(n))
    q = (qscale * torch.randn(N, HG + 3, c.d, generator=c.g)).to(c.dtype)
    if mutate:
        mutate(c, q)
    cache, st = c.device_cache(), _status()
    im = None
    if image:
        im = _image(c, cache)
        nexus.quantize(cache, im, st)
        if held is not None:
            im.rows.copy_(torch.as_tensor(held))
    qd = q.to(DEV)[:, 1:1 + HG]                                      # a strided view
    if packed_out:
        out = torch.full((N, HG, c.d), math.nan, dtype=c.dtype, device=DEV)
    else:
        out = torch.full((N, HG + 2, c.d), math.nan, dtype=c.dtype, device=DEV)[:, 1:-1]
    lse = torch.full((N, HG), math.nan, device=DEV)
    mt = max(max(n), 1)
    ws = nexus.alloc_attend_workspace(cache, tokens=N, max_tokens=mt)
    ws.fill_(0xFF)                                                   # it may hold anything
    torch.cuda.synchronize()
    kw = dict(max_tokens=mt, cu_tokens=None if uniform else c.cu(n).to(DEV), causal=causal,
              image=im, scale=scale)
    nexus.attend(cache, layer, qd, out, ws, st, lse=lse, **kw)
    out2 = torch.full((N, HG, c.d), math.nan, dtype=c.dtype, device=DEV)
    nexus.attend(cache, layer, qd, out2, ws, st, **kw)               # no lse, used workspace
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert torch.equal(out2, out)                                    # the same bits each time
    sc = c.d ** -0.5 if scale is None else scale
    worst, a = 0.0, 0
    codes8 = None if im is None else [x.cpu().float() for x in (im.k, im.v, im.k_scale, im.v_scale)]
    for s, m in enumerate(n):
        for h in range(c.H):
            T = int(c.lens[layer, s, h])
            at = c.at(layer, s, h, T)
            k, v = c.k[at].double(), c.v[at].double()
            if image:
                r = int(im.rows[layer, s, h])
                for t, qt, qs in ((k, codes8[0], codes8[2]), (v, codes8[1], codes8[3])):
                    codes = qt[c.at(layer, s, h, r)].double()
                    per = [float(qs[_scale_at(c, layer, s, h, j)]) for j in range(0, r, c.b)]
                    t[:r] = codes * torch.tensor(per, dtype=torch.float64).repeat_interleave(c.b)[:, None]
            rows = q[a:a + m, 1 + h * c.G:1 + (h + 1) * c.G].reshape(m * c.G, c.d)
            M = [(T - (m - 1 - i) if causal else T) for i in range(m) for _ in range(c.G)]
            ro, rl, A, big = attend64(rows, k, v, M, sc)
            got = out[a:a + m, h * c.G:(h + 1) * c.G].reshape(m * c.G, c.d).cpu().double()
            gl = lse[a:a + m, h * c.G:(h + 1) * c.G].reshape(-1).cpu().double()
            dx = abs(sc) * big * (2.0 ** -24 * (c.d + 8) if c.dtype == BF else 2.0 ** -20)
            p = (2.0 ** -11 + 2.0 ** -19 if image else 2.0 ** -8) if c.dtype == BF else 2.0 ** -19
            if image and int(im.rows[layer, s, h]) < T:
                p = 2.0 ** -8                                        # bf16 rows behind the image
            tol = HALF[c.dtype] * ro.abs() + (p + 2 * dx)[:, None] * A + 1e-30
            err = (got - ro).abs()
            assert torch.all(err <= tol), (s, h, float((err / tol).max()))
            none = torch.isinf(rl)
            assert torch.equal(none, torch.tensor([x <= 0 for x in M], dtype=torch.bool))
            assert torch.all(torch.isinf(gl[none])) and torch.all(gl[none] < 0)
            assert torch.all(got[none] == 0)
            el = (gl - rl).abs()[~none]
            assert torch.all(el <= (dx + 2.0 ** -19 * (1 + rl.abs()))[~none]), (s, h)
            if el.numel():
                worst = max(worst, float((err / tol).max()))
        a += m
    return worst


LENGTHS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 511, 700]


@pytest.mark.parametrize("kind", ["bf16", "bf16_64", "image", "image_64", "f32", "f32_64"])
@pytest.mark.parametrize("group", [1, 3, 4, 8])
def test_attend_one_token_over_every_length(kind, group):
    c = Case(seqs=len(LENGTHS), kv_heads=2, group=group, d=64 if kind.endswith("_64") else 128,
             dtype=F32 if kind.startswith("f32") else BF, capacity=701,
             lens=[[a, b] for a, b in zip(LENGTHS, reversed(LENGTHS))], seed=group)
    _check_attend(c, [1] * c.S, image=kind.startswith("image"), uniform=True)


@pytest.mark.parametrize("kind", ["bf16", "image", "f32"])
@pytest.mark.parametrize("page", [8, 16, 32, 64, 128])
def test_attend_paged_ragged_tokens(kind, page):
    c = Case(seqs=5, kv_heads=3, group=2, dtype=F32 if kind == "f32" else BF, page=page,
             capacity=300, lens=[[300, 1, 77], [20, 250, 3], [40, 40, 40], [5, 129, 64], [0, 17, 9]],
             seed=page)
    _check_attend(c, [4, 0, 20, 1, 9], image=kind == "image")


@pytest.mark.parametrize("kind", ["bf16", "bf16_64", "image", "image_64", "f32", "f32_64"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("tokens", [2, 5, 16, 33, 64, 130])
def test_attend_chunks(kind, causal, tokens):
    c = Case(seqs=2, kv_heads=2, group=3, d=64 if kind.endswith("_64") else 128,
             dtype=F32 if kind.startswith("f32") else BF, capacity=333,
             lens=[[333, 140], [tokens, max(1, tokens - 3)]], seed=tokens)
    _check_attend(c, [tokens, tokens - 1], causal=causal, image=kind.startswith("image"),
                  packed_out=tokens != 5)


@pytest.mark.parametrize("kind", ["bf16", "image", "f32"])
@pytest.mark.parametrize("group,tokens", [(1, 1), (8, 3), (16, 1), (5, 7), (32, 2), (64, 1), (1, 64)])
def test_attend_row_counts(kind, group, tokens):
    c = Case(seqs=2, kv_heads=1, group=group, dtype=F32 if kind == "f32" else BF, capacity=600,
             lens=[[600], [37]], seed=group)
    _check_attend(c, [tokens, tokens], image=kind == "image", uniform=True)


@pytest.mark.parametrize("kind", ["bf16", "image", "f32"])
def test_attend_long_slices_split(kind):
    c = Case(seqs=2, kv_heads=2, group=4, dtype=F32 if kind == "f32" else BF, capacity=20000,
             lens=[[20000, 4097], [12345, 0]], seed=9)
    _check_attend(c, [1, 1], image=kind == "image", uniform=True)
    _check_attend(c, [3, 40], image=kind == "image")


def test_attend_image_behind_the_cache():
    # the image stops at a block, the newest rows come from the cache; none held; all held
    c = Case(seqs=3, kv_heads=2, group=4, page=16, capacity=400, lens=[[400, 399], [100, 16], [33, 15]], seed=2)
    for held in ([[64, 0], [96, 16], [16, 0]], [[0, 0]] * 3, [[400, 384], [96, 16], [32, 0]]):
        _check_attend(c, [2, 1, 1], image=True, held=[held])


@pytest.mark.parametrize("kind", ["bf16", "image", "f32"])
def test_attend_peaked_and_far_logits(kind):
    # logits of hundreds, of both signs: one row carries a softmax, or all are far below 0
    def mutate(c, q):
        at = c.at(0, 0, 0, int(c.lens[0, 0, 0]))
        rows = c.k[at]
        rows[:, 0] = -8.0                                            # all far below ...
        rows[150, 0] = 30.0                                          # ... but one, late
        c.k[at] = rows
        q[..., 0] = 40.0
    c = Case(seqs=1, kv_heads=2, group=4, dtype=F32 if kind == "f32" else BF, capacity=300, lens=300, seed=4)
    _check_attend(c, [3], image=kind == "image", mutate=mutate)
    c = Case(seqs=1, kv_heads=2, group=4, dtype=F32 if kind == "f32" else BF, capacity=300, lens=300, seed=5)
    _check_attend(c, [2], image=kind == "image", scale=0.0)
    _check_attend(c, [2], image=kind == "image", scale=-0.3)
    _check_attend(c, [2], image=kind == "image", qscale=1e-3)


@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** 40])
@pytest.mark.parametrize("kind", ["bf16", "image", "f32"])
def test_attend_extreme_query_sizes(kind, size):
    # queries far outside the range of 16-bit floats, brought back by the scale
    c = Case(seqs=1, kv_heads=1, group=4, dtype=F32 if kind == "f32" else BF, capacity=100, lens=100, seed=6)
    _check_attend(c, [1], image=kind == "image", qscale=size, scale=1 / (11.3 * size))


def test_attend_layer_and_other_stream():
    c = Case(seqs=2, layers=3, kv_heads=2, group=2, capacity=64, lens=50, seed=8)
    _check_attend(c, [1, 2], layer=2)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        _check_attend(c, [1, 2], layer=1, image=True)


def test_attend_infinite_and_nan_rows_stay_in_their_slice():
    # an infinite key drops out (its logit is -inf); NaN shows in its own slice only
    c = Case(seqs=3, kv_heads=1, group=2, capacity=64, lens=40, seed=1)
    q = torch.rand(3, 2, 128, generator=c.g).to(BF) + 0.5            # positive
    c.k[c.at(0, 0, 0, 1)] = -math.inf
    c.v[0, 2, 0, 5] = math.nan
    cache, st = c.device_cache(), _status()
    out = torch.zeros(3, 2, 128, dtype=BF, device=DEV)
    ws = nexus.alloc_attend_workspace(cache, tokens=3, max_tokens=1)
    nexus.attend(cache, 0, q.to(DEV), out, ws, st, max_tokens=1)
    torch.cuda.synchronize()
    at = c.at(0, 0, 0, 40, 1)
    ref, _, A, _ = attend64(q[0], c.k[at], c.v[at], [39, 39], 128 ** -0.5)
    assert torch.all((out[0].cpu().double() - ref).abs() <= 2.0 ** -6 * A)
    assert torch.isfinite(out[1].float()).all() and torch.isnan(out[2].float()).all()


def test_attend_faults_are_flagged():
    c = Case(seqs=3, kv_heads=2, group=2, page=16, capacity=64, lens=[[40, 40], [50, 50], [60, 60]])
    cache, st = c.device_cache(), _status()
    q = torch.randn(3, 4, 128, generator=c.g).to(DEV, BF)
    out = torch.full_like(q, math.nan)
    ws = nexus.alloc_attend_workspace(cache, tokens=3, max_tokens=1)
    cache.lens[0, 0, 1], cache.lens[0, 1, 0] = -1, 65
    nexus.attend(cache, 0, q, out, ws, st, max_tokens=1)
    torch.cuda.synchronize()
    assert int(st.item()) == nexus.NX_DEV_BAD_LEN
    assert torch.all(out[0, 2:] == 0) and torch.all(out[1, :2] == 0)
    assert torch.isfinite(out.float()).all() and torch.all(out[2].float().abs().amax(-1) > 0)
    st.zero_()
    cache = c.device_cache()
    cache.block_table[1, 1] = c.pages                                # rows 16 .. 31 of sequence 1
    nexus.attend(cache, 0, q, out, ws, st, max_tokens=1)
    torch.cuda.synchronize()
    assert int(st.item()) == nexus.NX_DEV_BAD_PAGE
    keep = torch.cat([torch.arange(16), torch.arange(32, 50)])
    at = c.at(0, 1, 0, 50)
    ref, _, A, _ = attend64(q[1, :2].cpu(), c.k[at][keep], c.v[at][keep], [34, 34], 128 ** -0.5)
    assert torch.all((out[1, :2].cpu().double() - ref).abs() <= 2.0 ** -6 * A)
    st.zero_()
    cache = c.device_cache()
    im = _image(c, cache)
    nexus.quantize(cache, im, st)
    im.rows[0, 1, 0], im.rows[0, 2, 1] = 64, 8
    nexus.attend(cache, 0, q, out, ws, st, max_tokens=1, image=im)
    torch.cuda.synchronize()
    assert int(st.item()) == nexus.NX_DEV_BAD_IMAGE
    assert torch.all(out[1, :2] == 0) and torch.all(out[2, 2:] == 0)
    st.zero_()
    nexus.attend(cache, 0, q, out, ws, st, max_tokens=1,
                 cu_tokens=torch.tensor([0, 1, 0, 2], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert int(st.item()) == nexus.NX_DEV_BAD_TOKENS


def test_no_tokens_is_no_work():
    c = Case(seqs=2, kv_heads=2, group=2, capacity=32, lens=5)
    cache, st = c.device_cache(), _status()
    cu = torch.zeros(3, dtype=torch.int32, device=DEV)
    e = torch.empty(0, 4, 128, dtype=BF, device=DEV)
    kv = torch.empty(0, 2, 128, dtype=BF, device=DEV)
    ws = nexus.alloc_attend_workspace(cache, tokens=0, max_tokens=1)
    nexus.append(cache, 0, e, kv, kv, torch.empty(0, dtype=torch.int32, device=DEV), e, st,
                 max_tokens=1, cu_tokens=cu)
    nexus.attend(cache, 0, e, e, ws, st, max_tokens=1, cu_tokens=cu)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and torch.all(cache.lens == 5)


def test_decode_calls_replay_from_a_graph():
    c = Case(seqs=2, kv_heads=2, group=4, capacity=100, lens=[[40, 33], [64, 7]], seed=12)
    cache, st = c.device_cache(), _status()
    im = nexus.new_image(cache)
    rot = nexus.Rotary(_freqs(128), device=DEV)
    q, k, v = (torch.randn(2, h, 128, generator=c.g).to(DEV, BF) for h in (8, 2, 2))
    pos = torch.tensor([40, 64], dtype=torch.int32, device=DEV)
    qr, out = torch.empty_like(q), torch.empty_like(q)
    ws = nexus.alloc_attend_workspace(cache, tokens=2, max_tokens=1)

    def step():
        nexus.append(cache, 0, q, k, v, pos, qr, st, max_tokens=1, rotary=rot)
        nexus.quantize(cache, im, st)
        nexus.attend(cache, 0, qr, out, ws, st, max_tokens=1, image=im)

    saved = [t.clone() for t in (cache.k, cache.v, cache.pos, cache.lens, im.rows)]
    for _ in range(3):
        step()
    torch.cuda.synchronize()
    ref, ref_lens = out.clone(), cache.lens.clone()
    for t, o in zip((cache.k, cache.v, cache.pos, cache.lens, im.rows), saved):
        t.copy_(o)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert torch.equal(out, ref) and torch.equal(cache.lens, ref_lens)


# ---------------------------------------------------------------------------
# many query rows: pages, bounds, wide loops
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["bf16", "image"])
@pytest.mark.parametrize("page", [8, 16, 64, 128])
def test_attend_bad_page_under_many_rows(kind, page):
    # a page out of range is left out of every row's sums, whatever kernel takes the call
    c = Case(seqs=2, kv_heads=2, group=4, page=page, capacity=640, lens=[[640, 600], [300, 511]], seed=page)
    cache, st = c.device_cache(), _status()
    im = None
    if kind == "image":
        im = _image(c, cache)
        nexus.quantize(cache, im, st)
    which = 256 // page
    cache.block_table[0, which] = c.pages + 5
    n = 24                                                           # 96 rows per slice
    q = torch.randn(2 * n, 8, 128, generator=c.g).to(BF)
    out = torch.full((2 * n, 8, 128), math.nan, dtype=BF, device=DEV)
    ws = nexus.alloc_attend_workspace(cache, tokens=2 * n, max_tokens=n)
    nexus.attend(cache, 0, q.to(DEV), out, ws, st, max_tokens=n, image=im)
    torch.cuda.synchronize()
    assert int(st.item()) == nexus.NX_DEV_BAD_PAGE
    assert torch.isfinite(out.float()).all()
    for s in range(2):
        for h in range(2):
            T = int(c.lens[0, s, h])
            at = c.at(0, s, h, T)
            slots = torch.arange(T)
            good = (slots // page != which) if s == 0 else slots >= 0
            k, v = c.k[at][good].double(), c.v[at][good].double()
            rows = q[s * n:(s + 1) * n, h * 4:(h + 1) * 4].reshape(-1, 128)
            M = [int((slots[:T - (n - 1 - i)] >= 0)[good[:T - (n - 1 - i)]].sum())
                 for i in range(n) for _ in range(4)]
            ref, _, A, _ = attend64(rows, k, v, M, 128 ** -0.5)
            got = out[s * n:(s + 1) * n, h * 4:(h + 1) * 4].reshape(-1, 128).cpu().double()
            # the image's own rounding: half a step of e4m3, 2^-4, of keys and values
            tol = (2.0 ** -6 if im is None else 0.5) * A + 2.0 ** -8
            assert torch.all((got - ref).abs() <= tol), (s, h)


@pytest.mark.parametrize("kind", ["bf16", "image", "f32"])
def test_attend_bound_far_above_the_tokens(kind):
    # max_tokens is only a bound: 3 tokens under a bound of 2^30
    c = Case(seqs=3, kv_heads=2, group=2, dtype=F32 if kind == "f32" else BF, capacity=64, lens=40, seed=3)
    cache, st = c.device_cache(), _status()
    im = None
    if kind == "image":
        im = _image(c, cache)
        nexus.quantize(cache, im, st)
    cu = c.cu([1, 0, 2]).to(DEV)
    q = torch.randn(3, 4, 128, generator=c.g).to(DEV, c.dtype)
    a, b = torch.empty_like(q), torch.empty_like(q)
    ws = nexus.alloc_attend_workspace(cache, tokens=3, max_tokens=1 << 30)
    nexus.attend(cache, 0, q, a, ws, st, max_tokens=1 << 30, cu_tokens=cu, image=im)
    nexus.attend(cache, 0, q, b, ws, st, max_tokens=2, cu_tokens=cu, image=im)
    kv = torch.zeros(3, 2, 128, dtype=c.dtype, device=DEV)
    nexus.append(cache, 0, None, kv, kv, torch.zeros(3, dtype=torch.int32, device=DEV), None, st,
                 max_tokens=1 << 30, cu_tokens=cu)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert torch.equal(a, b)
    assert cache.lens[0].tolist() == [[41, 41], [40, 40], [42, 42]]


@pytest.mark.parametrize("kind", ["bf16", "image"])
@pytest.mark.parametrize("group,tokens", [(8, 17), (4, 64), (2, 129), (16, 40)])
def test_attend_many_rows_split_over_blocks(kind, group, tokens):
    # long slices of few sequences: every unit's pieces come from many thread blocks
    c = Case(seqs=1, kv_heads=2, group=group, capacity=6000, lens=[[6000, 4321]], seed=tokens)
    _check_attend(c, [tokens], image=kind == "image")
    _check_attend(c, [tokens], image=kind == "image", causal=False, scale=-0.05)


def test_attend_many_sequences_many_rows():
    # more units than thread blocks, ragged, some empty
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 200, (60, 3))
    c = Case(seqs=60, kv_heads=3, group=2, d=64, page=16, capacity=208, lens=lens, seed=1)
    n = rng.integers(0, 20, 60).tolist()
    _check_attend(c, n)
    _check_attend(c, n, image=True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [4, 16, 40, 200])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** -30, 2.0 ** 7, 2.0 ** 9, 2.0 ** 100, 0.7])
def test_attend_reads_every_code(d, group, scale):
    # equal keys and 32 equal value rows per block: the output is the value, code times scale,
    # for every finite code, below the normal range too (0.7: any scale will do)
    c = Case(seqs=4, kv_heads=1, group=group, d=d, capacity=64, lens=64, seed=1)
    cache, st = c.device_cache(), _status()
    cache.k.zero_()
    im = _image(c, cache)
    im.k.view(torch.uint8).zero_()
    codes = torch.arange(256, dtype=torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x35
    if d == 64:
        rows = codes.view(4, 64)
    else:
        rows = codes.view(2, 128).repeat(2, 1)
    im.v.view(torch.uint8)[0, :, 0] = rows[:, None].to(DEV)
    im.k_scale.fill_(1.0)
    im.v_scale.fill_(scale)
    im.rows.fill_(64)
    q = torch.randn(4, group, d, generator=c.g).to(DEV, BF)
    out = torch.full_like(q, math.nan)
    ws = nexus.alloc_attend_workspace(cache, tokens=4, max_tokens=1)
    nexus.attend(cache, 0, q, out, ws, st, max_tokens=1, image=im)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    want = rows.view(torch.float8_e4m3fn).double() * torch.tensor(scale, dtype=torch.float32).double()
    # 64 equal probabilities: sums of equal terms; a scale that is no power of two is rounded
    # with its values once more
    err = (out.cpu().double() - want[:, None]).abs()
    assert torch.all(err <= (2.0 ** -16 if scale != 0.7 else 2.0 ** -7) * want[:, None].abs())


@pytest.mark.parametrize("group", [4, 16, 40])
def test_attend_nan_codes_give_nan(group):
    c = Case(seqs=2, kv_heads=1, group=group, capacity=64, lens=64, seed=1)
    c.v[0, 1, 0, 7, 3] = math.nan
    cache, st = c.device_cache(), _status()
    im = _image(c, cache)
    nexus.quantize(cache, im, st)
    q = torch.randn(2, group, 128, generator=c.g).to(DEV, BF)
    out = torch.zeros_like(q)
    ws = nexus.alloc_attend_workspace(cache, tokens=2, max_tokens=1)
    nexus.attend(cache, 0, q, out, ws, st, max_tokens=1, image=im)
    torch.cuda.synchronize()
    bad = torch.isnan(out.float())
    assert not bad[0].any() and bad[1, :, 3].all() and not bad[1, :, :3].any() and not bad[1, :, 4:].any()


CUTS = [0, 1, 8, 63, 64, 65, 128, 129, 191, 300, 447, 449, 511, 513, 800, 899, 900]


@pytest.mark.parametrize("kind", ["bf16", "bf16_64", "image", "image_64", "f32", "f32_64"])
@pytest.mark.parametrize("seqs,capacity,one", [
    (2, 900, True), (5, 2000, False), (20, 900, False), (20, 2001, False), (40, 500, False),
    (45, 900, False), (60, 450, True), (120, 512, True)])
def test_attend_blocks_per_slice(kind, seqs, capacity, one):
    # a block, a cluster of 8, 4 or 2 blocks, or an even share per slice, by the number of slices
    # and their capacity; fewer tiles than blocks, none, and rows that see none of a block's
    group = 4
    c = Case(seqs=seqs, kv_heads=2, group=group, d=64 if kind.endswith("_64") else 128,
             dtype=F32 if kind.startswith("f32") else BF, capacity=capacity,
             lens=[[min(capacity, CUTS[i % 17]), min(capacity, CUTS[(7 * i + 3) % 17]) if i else capacity]
                   for i in range(seqs)], seed=seqs)
    _check_attend(c, [1] * seqs, image=kind.startswith("image"), uniform=True)
    if one and not kind.startswith("f32"):
        assert nexus.last_launch_names() == ["attend"]
    n = [(3 * i + 1) % 5 for i in range(seqs)]
    _check_attend(c, n, image=kind.startswith("image"))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [1, 5, 30])
@pytest.mark.parametrize("at", [0, 63, 64, 700])
def test_attend_nan_and_infinite_rows_among_the_blocks_of_a_slice(kind, tokens, at):
    # a NaN key or value reaches every row of its slice and no other slice; an infinite key
    # drops out; an infinite value makes infinities or NaN
    dt = F32 if kind == "f32" else BF
    c = Case(seqs=5, kv_heads=1, group=2, dtype=dt, capacity=701, lens=701, seed=at)
    q = (torch.rand(5 * tokens, 2, 128, generator=c.g) + 0.5).to(dt)  # positive
    c.k[0, 0, 0, at] = -math.inf
    c.v[0, 1, 0, at] = math.nan
    c.k[0, 2, 0, at] = math.nan
    c.v[0, 4, 0, at] = math.inf
    cache, st = c.device_cache(), _status()
    out = torch.zeros(5 * tokens, 2, 128, dtype=dt, device=DEV)
    ws = nexus.alloc_attend_workspace(cache, tokens=5 * tokens, max_tokens=tokens)
    nexus.attend(cache, 0, q.to(DEV), out, ws, st, max_tokens=tokens, causal=False)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    if tokens == 1:
        assert nexus.last_launch_names() == ["attend"]
    out = out.reshape(5, tokens * 2, 128).cpu()
    keep = torch.tensor([j for j in range(701) if j != at])
    ref, _, A, _ = attend64(q[:tokens].reshape(-1, 128), c.k[0, 0, 0][keep], c.v[0, 0, 0][keep],
                            [700] * (2 * tokens), 128 ** -0.5)
    assert torch.all((out[0].double() - ref).abs() <= 2.0 ** -6 * A)
    nan = torch.isnan(out)
    assert not nan[0].any() and nan[1].all() and nan[2].all() and not nan[3].any()
    assert not torch.isfinite(out[4]).any()
