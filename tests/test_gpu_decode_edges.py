"""nexus_append, nexus_quantize and nexus_attend where one call's parts meet: pieces that share a
block's memory, scales that differ within a slice, rows that are taken back. Tolerances as in
test_gpu_decode.py."""
import math

import numpy as np
import pytest
import torch

from decode_harness import DEV, Case, attend64
from streaming_kv_cache_step_gb300 import nexus
from test_gpu_decode import BF, F32, _check_attend, _image, _scale_at, _status  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("tokens", [9, 32])
def test_attend_pieces_of_one_block_follow_one_another(d, page, tokens):
    # one row tile per slice and several slices per thread block: a slice's outputs pass through
    # the shared memory that the next one's whole tiles of K and V are copied to
    rng = np.random.default_rng(tokens + page)
    c = Case(seqs=60, kv_heads=4, group=4, d=d, page=page, capacity=384,
             lens=rng.choice([64, 128, 192, 256, 320, 384], (60, 4)), seed=page)
    _check_attend(c, [tokens] * 60, uniform=True)


# ---------------------------------------------------------------------------
# attend from an image whose blocks differ in scale
# ---------------------------------------------------------------------------

def _by_block(c, powers, name="v"):
    """Multiplies a slice's blocks by powers of two (None: zeros), in turn, in every slice."""
    t = getattr(c, name)
    for s in range(c.S):
        for h in range(c.H):
            T = int(c.lens[0, s, h])
            for i, j in enumerate(range(0, T, c.b)):
                p = powers[(i + s + h) % len(powers)]
                at = c.at(0, s, h, min(T, j + c.b), j)
                t[at] = t[at] * 2.0 ** p if p is not None else 0.0


@pytest.mark.parametrize("page", [0, 8, 16, 64])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group,tokens", [(4, 1), (16, 1), (5, 9)])
@pytest.mark.parametrize("powers", [[None, -24, -24, -24], [None, -30, 20], [-70, 40, -9, -10, 0],
                                    [None, -50, -50, -50, -50, -50, -50], [0, 7, 0, 9, -8]],
                         ids=["zeros", "mixed", "far", "tiny", "near"])
def test_attend_image_scales_differ_within_a_slice(powers, group, tokens, d, page):
    # a block's scale is its own: next to zeros (their scale is 1) or to values 2^50 times its own,
    # its codes come out as exactly as alone, wherever the weights lie
    c = Case(seqs=2, kv_heads=2, group=group, d=d, page=page, capacity=704,
             lens=[[704, 640], [96, 352]], seed=len(powers))
    _by_block(c, powers)
    _check_attend(c, [tokens] * 2, image=True, uniform=True)


@pytest.mark.parametrize("page", [0, 8])
@pytest.mark.parametrize("group", [4, 16])
@pytest.mark.parametrize("less", [24.0, 30.0, 40.0, 100.0])
def test_attend_image_large_values_with_small_weights(less, group, page):
    # values 2^40 times the others', at logits that leave them a small part (e^-24 2^40 = 41), an
    # even part or nothing of the sum, block by block: both sides of it show in the output
    c = Case(seqs=1, kv_heads=2, group=group, page=page, capacity=512, lens=512, seed=7)
    for h in range(2):
        for j in range(0, 512, 2 * c.b):
            at = c.at(0, 0, h, j + c.b, j)
            c.v[at] = c.v[at] * 2.0 ** 40
            c.k[at][..., 0] = 0.0
            k = c.k[at]
            k[:, 0] = -less
            c.k[at] = k
        for j in range(c.b, 512, 2 * c.b):
            at = c.at(0, 0, h, j + c.b, j)
            k = c.k[at]
            k[:, 0] = 0.0
            c.k[at] = k

    def mutate(c, q):
        q[..., 0] = 128 ** 0.5                                       # times the scale: 1

    _check_attend(c, [1], image=True, mutate=mutate)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group,tokens", [(1, 8), (2, 8), (4, 10), (8, 10)])
def test_attend_image_large_values_that_are_not_seen_yet(group, tokens, d):
    # the newest rows, 2^40 and 2^100 times the others, stand in the image but most tokens do not
    # see them
    for up in (40, 100):
        c = Case(seqs=2, kv_heads=2, group=group, d=d, page=8, capacity=256, lens=[[256, 128], [64, 8]],
                 seed=up)
        for s in range(2):
            for h in range(2):
                T = int(c.lens[0, s, h])
                at = c.at(0, s, h, T, T - 8)
                c.v[at] = c.v[at] * 2.0 ** up
        _check_attend(c, [tokens] * 2, image=True, uniform=True)


# ---------------------------------------------------------------------------
# an image of rows that are taken back
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("page", [0, 8, 64])
@pytest.mark.parametrize("in_place", [False, True], ids=["lens_in", "lens"])
@pytest.mark.parametrize("tokens", [6, 40])
def test_append_takes_drafts_back_from_an_image(page, in_place, tokens):
    # drafts that stood in full blocks of the image are replaced: their codes are read no more, the
    # blocks before them are, and other layers keep theirs
    c = Case(seqs=3, kv_heads=2, group=2, layers=2, page=page, capacity=192,
             lens=[[27, 60], [32, 31], [64, 5]], seed=tokens)
    cache, st = c.device_cache(), _status()
    im = nexus.new_image(cache)
    new = lambda: [torch.randn(3 * tokens, h, 128, generator=c.g).to(DEV, BF) for h in (4, 2, 2)]  # noqa: E731
    pos = torch.arange(3 * tokens, dtype=torch.int32, device=DEV)
    base = cache.lens[1].clone()
    base[0, 0] += 2                                                  # two drafts are good
    q, k, v = new()
    out = torch.empty_like(q)
    nexus.append(cache, 1, q, k, v, pos, out, st, max_tokens=tokens)
    nexus.quantize(cache, im, st)
    held = im.rows.clone()
    if in_place:
        cache.lens[1] = base
    q, k, v = new()
    nexus.append(cache, 1, q, k, v, pos, q, st, max_tokens=tokens, image=im,
                 lens_in=None if in_place else base)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and torch.equal(cache.lens[1], base + tokens)
    want = held.clone()
    want[1] = torch.minimum(held[1], base // c.b * c.b)
    assert torch.equal(im.rows, want) and not torch.equal(want, held)
    # a new image that holds the same rows gives the same bits
    fresh = nexus.new_image(cache)
    nexus.quantize(cache, fresh, st)
    fresh.rows.copy_(im.rows)
    outs = []
    ws = nexus.alloc_attend_workspace(cache, tokens=3 * tokens, max_tokens=tokens)
    for x in (im, fresh):
        outs.append(torch.full_like(q, math.nan))
        nexus.attend(cache, 1, q, outs[-1], ws, st, max_tokens=tokens, image=x)
    # and brought up to date it is the one that was made from nothing
    nexus.quantize(cache, im, st)
    nexus.quantize(cache, fresh, st)
    for x in (im, fresh):
        outs.append(torch.full_like(q, math.nan))
        nexus.attend(cache, 1, q, outs[-1], ws, st, max_tokens=tokens, image=x)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and torch.equal(im.rows, cache.lens // c.b * c.b)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[2], outs[3])


def test_append_leaves_the_image_of_a_slice_that_takes_nothing():
    # no room, a bad length, bad token ranges: the slice stays, and so does what the image holds
    c = Case(seqs=2, kv_heads=2, group=1, page=8, capacity=64, lens=[[40, 64], [40, 40]], seed=1)
    cache, st = c.device_cache(), _status()
    im = nexus.new_image(cache)
    nexus.quantize(cache, im, st)
    x = torch.ones(6, 2, 128, dtype=BF, device=DEV)
    pos = torch.zeros(6, dtype=torch.int32, device=DEV)
    before = torch.tensor([[[20, 62], [-1, 20]]], dtype=torch.int32, device=DEV)
    nexus.append(cache, 0, None, x, x, pos, None, st, max_tokens=3, lens_in=before[0], image=im)
    torch.cuda.synchronize()
    assert int(st.item()) == nexus.NX_DEV_FULL | nexus.NX_DEV_BAD_LEN
    assert im.rows[0].tolist() == [[16, 64], [40, 16]]
    st.zero_()
    nexus.append(cache, 0, None, x, x, pos, None, st, max_tokens=3, lens_in=before[0] * 0, image=im,
                 cu_tokens=torch.tensor([0, 6, 6], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert int(st.item()) == nexus.NX_DEV_BAD_TOKENS
    assert im.rows[0].tolist() == [[16, 64], [0, 0]]


@pytest.mark.parametrize("kind", ["bf16", "bf16_64", "image", "image_64", "f32", "f32_64"])
@pytest.mark.parametrize("tokens", [1, 5, 12])
@pytest.mark.parametrize("size", [1e36, 1e-30])
def test_attend_values_near_the_end_of_the_range(kind, tokens, size):
    # finite values whose weighted sums are finite come out finite: 100 rows of 10^36
    c = Case(seqs=2, kv_heads=2, group=4, d=64 if kind.endswith("_64") else 128,
             dtype=F32 if kind.startswith("f32") else BF, capacity=104, lens=[[104, 96], [33, 70]], seed=3)
    c.v *= size
    _check_attend(c, [tokens] * 2, image=kind.startswith("image"), uniform=True)


# ---------------------------------------------------------------------------
# pages out of range, held to the tolerances of whole slices
# ---------------------------------------------------------------------------

def _check_bad_pages(c, n, bad, image, held=None, causal=True):
    """Pages bad[s] (indexes into the sequence's table) of sequence s are out of range: their slots
    count for nothing, in the output and in lse."""
    HG, N = c.H * c.G, int(sum(n))
    q = torch.randn(N, HG, c.d, generator=c.g).to(c.dtype)
    cache, st = c.device_cache(), _status()
    im = None
    if image:
        im = _image(c, cache)
        nexus.quantize(cache, im, st)
        if held is not None:
            im.rows.copy_(torch.as_tensor(held))
    for s, pages in enumerate(bad):
        for i, p in enumerate(pages):
            cache.block_table[s, p] = (-1, c.pages, 1 << 30)[i % 3]
    out = torch.full((N, HG, c.d), math.nan, dtype=c.dtype, device=DEV)
    lse = torch.full((N, HG), math.nan, device=DEV)
    ws = nexus.alloc_attend_workspace(cache, tokens=N, max_tokens=max(n))
    ws.fill_(0xFF)
    nexus.attend(cache, 0, q.to(DEV), out, ws, st, max_tokens=max(n), cu_tokens=c.cu(n).to(DEV),
                 causal=causal, lse=lse, image=im)
    torch.cuda.synchronize()
    assert int(st.item()) == nexus.NX_DEV_BAD_PAGE
    sc, a = c.d ** -0.5, 0
    deq = None if im is None else [x.cpu().float() for x in (im.k, im.v, im.k_scale, im.v_scale)]
    for s, m in enumerate(n):
        for h in range(c.H):
            T = int(c.lens[0, s, h])
            at = c.at(0, s, h, T)
            k, v = c.k[at].double(), c.v[at].double()
            if image:
                r = int(im.rows[0, s, h])
                for t, codes, scales in ((k, deq[0], deq[2]), (v, deq[1], deq[3])):
                    per = [float(scales[_scale_at(c, 0, s, h, j)]) for j in range(0, r, c.b)]
                    t[:r] = codes[c.at(0, s, h, r)].double() * \
                        torch.tensor(per, dtype=torch.float64).repeat_interleave(c.b)[:, None]
            good = ~torch.isin(torch.arange(T) // c.page, torch.tensor(bad[s], dtype=torch.long))
            M = [int(good[:max(0, T - (m - 1 - i if causal else 0))].sum())
                 for i in range(m) for _ in range(c.G)]
            rows = q[a:a + m, h * c.G:(h + 1) * c.G].reshape(m * c.G, c.d)
            ro, rl, A, big = attend64(rows, k[good], v[good], M, sc)
            got = out[a:a + m, h * c.G:(h + 1) * c.G].reshape(m * c.G, c.d).cpu().double()
            gl = lse[a:a + m, h * c.G:(h + 1) * c.G].reshape(-1).cpu().double()
            dx = sc * big * (2.0 ** -24 * (c.d + 8) if c.dtype == BF else 2.0 ** -20)
            p = 2.0 ** -8 if c.dtype == BF else 2.0 ** -19
            if image and int(im.rows[0, s, h]) == T:
                p = 2.0 ** -11 + 2.0 ** -19
            half = 2.0 ** -8 if c.dtype == BF else 2.0 ** -24
            tol = half * ro.abs() + (p + 2 * dx)[:, None] * A + 1e-30
            assert torch.all((got - ro).abs() <= tol), (s, h)
            some = torch.tensor([x > 0 for x in M], dtype=torch.bool)
            assert torch.all(gl[~some] == -math.inf) and torch.all(got[~some] == 0)
            assert torch.all((gl - rl).abs()[some] <= (dx + 2.0 ** -19 * (1 + rl.abs()))[some]), (s, h)
        a += m


@pytest.mark.parametrize("kind", ["bf16", "image", "f32"])
@pytest.mark.parametrize("page", [8, 16, 32, 128])
@pytest.mark.parametrize("group,tokens", [(4, 1), (4, 4), (4, 10), (8, 12), (4, 60)])
def test_attend_leaves_bad_pages_out(kind, page, group, tokens):
    # 4 to 240 query rows per slice; a bad page in the middle, two in a row at an odd place, the first
    # and the last ones, and every page of a sequence
    per = 512 // page
    c = Case(seqs=5, kv_heads=2, group=group, dtype=F32 if kind == "f32" else BF, page=page, capacity=512,
             lens=[[512, 480], [300, 511], [256, 129], [512, 77], [130, 64]], seed=page + tokens)
    bad = [[per // 2], [1, 2], [0, 256 // page - 1], [per - 1], list(range(per))]
    _check_bad_pages(c, [tokens, 1, tokens, tokens, tokens], bad, kind == "image")
    if kind == "image":            # some of them among the rows behind the image
        held = [[[256, 480 // c.b * c.b], [32, 0], [128, 128], [480, 64], [0, 64]]]
        _check_bad_pages(c, [tokens, 1, tokens, tokens, tokens], bad, True, held=held, causal=False)


# ---------------------------------------------------------------------------
# values that are not finite in rows that only some tokens see
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["bf16", "bf16_64", "image", "image_64", "f32", "f32_64"])
@pytest.mark.parametrize("page", [0, 8])
@pytest.mark.parametrize("group,tokens", [(1, 2), (4, 2), (2, 7), (4, 10), (8, 12), (4, 60), (1, 300)])
def test_attend_values_that_are_not_finite_show_where_they_are_seen(kind, page, group, tokens):
    # infinities and NaN in single features of the newest rows: in tokens before them the same
    # features are finite and exact, in tokens that see them not finite
    d = 64 if kind.endswith("_64") else 128
    image, dt = kind.startswith("image"), F32 if kind.startswith("f32") else BF
    c = Case(seqs=3, kv_heads=2, group=group, d=d, dtype=dt, page=page, capacity=720,
             lens=[[720, 700], [tokens + 5, tokens], [320, 449]], seed=tokens)
    n = [tokens, max(1, tokens - 1), tokens]
    marks = (math.nan, math.nan) if image else (math.nan, math.inf, -math.inf)  # (codes hold no infinity)
    for s in range(c.S):
        for h in range(c.H):
            T = int(c.lens[0, s, h])
            for j, back in enumerate((0, 1, n[s] // 2, n[s] - 1)[:max(1, n[s])]):
                at = c.at(0, s, h, T - back, T - back - 1)
                rows = c.v[at]
                rows[:, (17 * j + 5 * h) % d] = marks[(j + s) % len(marks)]
                c.v[at] = rows
    HG, N = c.H * group, sum(n)
    q = torch.randn(N, HG, d, generator=c.g).to(dt)
    cache, st = c.device_cache(), _status()
    im = None
    if image:
        im = _image(c, cache)
        nexus.quantize(cache, im, st)
        im.rows[0, 2, 1] = 448 if tokens > 1 else im.rows[0, 2, 1]
    out = torch.zeros(N, HG, d, dtype=dt, device=DEV)
    lse = torch.zeros(N, HG, device=DEV)
    ws = nexus.alloc_attend_workspace(cache, tokens=N, max_tokens=max(n))
    kw = dict(max_tokens=max(n), cu_tokens=c.cu(n).to(DEV), image=im)
    nexus.attend(cache, 0, q.to(DEV), out, ws, st, lse=lse, **kw)
    out2 = torch.zeros_like(out)
    nexus.attend(cache, 0, q.to(DEV), out2, ws, st, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert torch.equal(out.nan_to_num(), out2.nan_to_num())
    deq = None if im is None else [x.cpu().float() for x in (im.k, im.v, im.k_scale, im.v_scale)]
    a, sc, seen = 0, d ** -0.5, 0
    for s, m in enumerate(n):
        for h in range(c.H):
            T = int(c.lens[0, s, h])
            at = c.at(0, s, h, T)
            k, v = c.k[at].double(), c.v[at].double()
            r = int(im.rows[0, s, h]) if image else 0
            if r:
                for t, codes, scales in ((k, deq[0], deq[2]), (v, deq[1], deq[3])):
                    per = [float(scales[_scale_at(c, 0, s, h, j)]) for j in range(0, r, c.b)]
                    t[:r] = codes[c.at(0, s, h, r)].double() * \
                        torch.tensor(per, dtype=torch.float64).repeat_interleave(c.b)[:, None]
            M = [T - (m - 1 - i) for i in range(m) for _ in range(group)]
            rows = q[a:a + m, h * group:(h + 1) * group].reshape(m * group, d)
            ro, rl, A, big = attend64(rows, k, v, M, sc)
            got = out[a:a + m, h * group:(h + 1) * group].reshape(m * group, d).cpu().double()
            gl = lse[a:a + m, h * group:(h + 1) * group].reshape(-1).cpu().double()
            fin = torch.isfinite(ro)
            assert torch.equal(torch.isfinite(got), fin), (s, h)
            dx = sc * big * (2.0 ** -24 * (d + 8) if dt == BF else 2.0 ** -20)
            p = 2.0 ** -8 if dt == BF else 2.0 ** -19
            tol = (2.0 ** -8 if dt == BF else 2.0 ** -24) * ro.abs() + (p + 2 * dx)[:, None] * A + 1e-30
            assert torch.all((got - ro).abs()[fin] <= tol[fin]), (s, h)
            some = torch.tensor(M) > 0
            assert torch.all((gl - rl).abs()[some] <= (dx + 2.0 ** -19 * (1 + rl.abs()))[some]), (s, h)
            seen += int((~fin).sum())
        a += m
    assert seen > 0


# ---------------------------------------------------------------------------
# whole prompts, and caches that hold far fewer rows than they could
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["bf16", "image", "f32"])
@pytest.mark.parametrize("page", [0, 16])
def test_attend_whole_prompts(kind, page):
    # every row of the slices is a token of the call: the causal triangle, and prompts of other lengths
    c = Case(seqs=3, kv_heads=2, group=2, dtype=F32 if kind == "f32" else BF, page=page, capacity=2112,
             lens=[[2100, 2100], [1, 1], [777, 777]], seed=page)
    _check_attend(c, [2100, 1, 777], image=kind == "image")


@pytest.mark.parametrize("kind", ["bf16", "image", "f32"])
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("tokens", [1, 5, 40])
def test_attend_few_rows_of_a_large_capacity(kind, page, tokens):
    # kernels are chosen by capacity: slices of any length give the same whatever it is
    c = Case(seqs=2, kv_heads=2, group=4, dtype=F32 if kind == "f32" else BF, page=page, capacity=1 << 15,
             lens=[[40, 1638], [257, 64]], seed=tokens)
    _check_attend(c, [tokens] * 2, image=kind == "image", uniform=True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [0, 8])
@pytest.mark.parametrize("tokens", [12, 40])
def test_attend_many_rows_over_scales_that_differ(tokens, page, d):
    # the kernel for more than 80 rows: zeros, 2^-70 to 2^40, and values near the end of the range
    for powers in ([None, -30, 20], [-70, 40, -9, -10, 0], [118, 110]):
        c = Case(seqs=2, kv_heads=2, group=8, d=d, page=page, capacity=256, lens=[[256, 192], [96, 70]],
                 seed=tokens)
        _by_block(c, powers)
        _check_attend(c, [tokens] * 2, image=True, uniform=True)
