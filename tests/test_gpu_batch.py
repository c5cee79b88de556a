"""nexus_plan, nexus_verify and nexus_attend_shared on the GPU against plain forms, and a serving
loop of them.

plan and verify give whole numbers: they are equal. attend_shared has the roundings of
nexus_attend, in units of what rounds (half a step of bf16 is 2^-8 of a value, of fp32 2^-24): the
output's (2^-8 or 2^-24 of it), the weights' (2^-8 of sum p |v| / sum p for bf16 rows; the image's
2^-11 or less is below that; fp32 rows 2^-19), what an error dx of the logits changes (2 dx of the
same sum; dx <= 2^-24 (d + 8) scale sum |q_i k_i| for exact products summed in fp32, 2^-20 scale sum
|q_i k_i| for fp32 rows), and where the two parts meet an exponential (2^-22) and some four fp32
roundings: 2^-20. lse errs by dx and the fp32 roundings of two sums and a join (2^-18)."""
import math

import numpy as np
import pytest
import torch

import batch_harness as B
from decode_harness import DEV, Case, attend64, rotate64
from streaming_kv_cache_step_gb300 import nexus

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def _status():
    return nexus.new_status(torch.device(DEV))


def _ints(x):
    return torch.as_tensor(np.ascontiguousarray(x).astype(np.int32), device=DEV)


def _bare_cache(layers=1, seqs=1, kv_heads=1, capacity=64, page=0, num_pages=0, table=None,
                lens=None):
    """A cache whose keys and values nobody looks at."""
    some = torch.zeros(64, dtype=BF, device=DEV)
    lens = torch.zeros(layers, seqs, kv_heads, dtype=torch.int32, device=DEV) if lens is None \
        else lens
    return nexus.Cache(k=some, v=some, pos=some.int(), lens=lens, layers=layers, seqs=seqs,
                       kv_heads=kv_heads, group=1, head_dim=64, capacity=capacity, page_size=page,
                       num_pages=num_pages, max_pages_per_seq=capacity // page if page else 0,
                       block_table=table)


# ---------------------------------------------------------------------------
# plan
# ---------------------------------------------------------------------------

class Pool:
    """The same tables twice: numpy's for the plain form, the GPU's for the call."""

    def __init__(self, layers, seqs, kv_heads, page, per, num_pages, rng):
        self.L, self.S, self.H, self.page, self.per, self.pages = (layers, seqs, kv_heads, page, per,
                                                                   num_pages)
        self.rng = rng
        self.capacity = per * page
        self.lens = np.zeros((layers, seqs, kv_heads), np.int64)
        self.table = rng.integers(-5, num_pages + 5, (seqs, per))
        self.held = np.zeros(seqs, np.int64)
        self.free = rng.permutation(num_pages)
        self.count = num_pages
        self.dev = dict(lens=_ints(self.lens), table=_ints(self.table), held=_ints(self.held),
                        free=_ints(self.free), count=_ints([num_pages]))
        self.cache = _bare_cache(layers, seqs, kv_heads, self.capacity, page, num_pages,
                                 self.dev["table"], self.dev["lens"])
        self.pool = nexus.Pool(free_pages=self.dev["free"], free_count=self.dev["count"],
                               held=self.dev["held"])

    def put(self):
        self.dev["lens"].copy_(_ints(self.lens))

    def call(self, n, tokens, max_tokens, first_pos, **kw):
        st = _status()
        cu = torch.full((self.S + 1,), -9, dtype=torch.int32, device=DEV)
        seq = torch.full((tokens,), -9, dtype=torch.int32, device=DEV)
        pos = torch.full((tokens,), -9, dtype=torch.int32, device=DEV)
        nexus.plan(self.cache, self.pool, _ints(n), cu, st, max_tokens=max_tokens, token_seq=seq,
                   token_pos=pos, first_pos=_ints(first_pos), **kw)
        torch.cuda.synchronize()
        assert nexus.last_launch_names() == ["plan"]
        return cu.cpu().tolist(), seq.cpu().tolist(), pos.cpu().tolist(), int(st.item())

    def plain(self, n, tokens, max_tokens, first_pos):
        cu, seq, pos, self.count, status = B.plan_plain(
            self.lens, n, self.capacity, tokens=tokens, max_tokens=max_tokens, page=self.page,
            num_pages=self.pages, table=self.table, free=self.free, count=self.count,
            held=self.held, first_pos=first_pos)
        pad = [-9] * (tokens - len(seq))
        return cu, seq + pad, pos + pad, status

    def check(self, n, tokens, max_tokens, first_pos):
        got = self.call(n, tokens, max_tokens, first_pos)
        want = self.plain(n, tokens, max_tokens, first_pos)
        assert got[3] == want[3], (got[3], want[3])
        assert got[0] == want[0] and got[1] == want[1] and got[2] == want[2]
        for name, mine in (("lens", self.lens), ("table", self.table), ("held", self.held),
                           ("free", self.free), ("count", [self.count])):
            assert np.array_equal(self.dev[name].cpu().numpy(), mine), name
        return want

    def disjoint(self):
        mine = [p for s in range(self.S) for p in self.table[s, :self.held[s]]]
        every = sorted(mine + list(self.free[:self.count]))
        assert every == list(range(self.pages))


@pytest.mark.parametrize("layers,seqs,kv_heads,page,per,share", [
    (1, 1, 1, 8, 4, 1.0), (2, 3, 2, 8, 9, 1.0), (3, 33, 5, 16, 20, 0.5), (32, 16, 8, 16, 64, 0.8),
    (1, 300, 8, 32, 12, 0.6), (7, 1025, 3, 64, 6, 0.7), (1, 8192, 1, 128, 3, 0.5),
    # pools so small that sequences wait for pages, too
    (3, 33, 5, 16, 20, 0.2), (1, 301, 8, 32, 12, 0.25), (7, 1023, 3, 64, 6, 0.3)])
def test_plan_over_many_steps(layers, seqs, kv_heads, page, per, share):
    # tokens arrive, evictions shorten slices, sequences end and come back
    rng = np.random.default_rng([layers, seqs, page])
    p = Pool(layers, seqs, kv_heads, page, per, max(per, int(seqs * per * share)), rng)
    most = p.capacity // 2 + 3
    seen = 0
    for step in range(12):
        n = rng.integers(0, most, seqs)
        n[rng.random(seqs) < 0.3] = 1
        n[rng.random(seqs) < 0.1] = 0
        n[rng.random(seqs) < 0.15] = -int(rng.integers(1, 5))
        tokens = int(np.maximum(n, 0).sum() * (0.6 if step % 4 == 3 else 1.0)) + step % 2
        cu, _, _, status = p.check(n, tokens, most if step % 3 else max(1, most - 4),
                                   rng.integers(-5, 1 << 30, seqs))
        p.disjoint()
        seen |= status
        grown = np.diff(cu)
        p.lens += grown[None, :, None]
        # every slice is evicted to a length of its own
        cut = rng.random(seqs) < 0.3
        p.lens[:, cut] = p.lens[:, cut] * rng.integers(1, 9, p.lens[:, cut].shape) // 8
        p.put()
    if share < 0.5:
        assert seen & B.NO_PAGES and seen & B.BAD_TOKENS and seen & B.FULL


@pytest.mark.parametrize("seqs", [1, 40, 1500])
def test_plan_repeats_with_held_in_and_free_count_in(seqs):
    rng = np.random.default_rng(seqs)
    p = Pool(2, seqs, 2, 16, 8, seqs * 8 + 3, rng)
    for _ in range(2):
        n = rng.integers(1, 60, seqs)
        cu = p.check(n, int(n.sum()), 60, [0] * seqs)[0]
        p.lens += np.diff(cu)[None, :, None]
        p.lens = p.lens * rng.integers(2, 5, p.lens.shape) // 4
        p.put()
    held, count = p.dev["held"].clone(), p.dev["count"].clone()
    n = rng.integers(-1, 60, seqs)
    free0, lens0 = p.dev["free"].clone(), p.dev["lens"].clone()
    first = p.call(n, 60 * seqs, 60, [5] * seqs, held_in=held, free_count_in=count)
    tables = [p.dev[k].clone() for k in ("table", "free", "held", "count", "lens")]
    again = p.call(n, 60 * seqs, 60, [5] * seqs, held_in=held, free_count_in=count)
    assert first == again
    assert all(torch.equal(a, p.dev[k])
               for a, k in zip(tables, ("table", "free", "held", "count", "lens")))
    # and in place the same
    p.dev["held"].copy_(held)
    p.dev["count"].copy_(count)
    p.dev["free"].copy_(free0)
    p.dev["lens"].copy_(lens0)
    p.check(n, 60 * seqs, 60, [5] * seqs)


def test_plan_refusals_one_by_one():
    rng = np.random.default_rng(3)
    p = Pool(2, 6, 2, 8, 10, 70, rng)
    p.check([20] * 6, 120, 20, [0] * 6)
    p.lens[:] = 20
    p.lens[1, 1, 0] = 81                                   # beyond capacity
    p.lens[0, 2, 1] = -1
    p.put()
    p.check([1, 1, 1, 61, 1, 1], 6, 80, [0] * 6)           # 20 + 61 is above capacity
    p.lens[:, 1:3] = 20
    p.put()
    p.check([1, 9, 1, 1, 0, 1], 5, 8, [0] * 6)             # 9 is above max_tokens
    p.held[4] = 11                                         # out of range, ending or not
    p.dev["held"].copy_(_ints(p.held))
    p.check([1, 1, 1, 1, 1, 1], 6, 8, [0] * 6)
    p.check([1, 1, 1, 1, -1, 1], 6, 8, [0] * 6)
    assert p.lens[:, 4].min() == 20
    p.held[4] = -2
    p.dev["held"].copy_(_ints(p.held))
    p.check([1, 1, 1, 1, -1, 1], 6, 8, [0] * 6)
    assert p.lens[:, 4].min() == 20
    # a slice of a sequence that ends may hold any length
    p.lens[0, 0, 0] = -7
    p.put()
    p.check([-1, 0, 0, 0, 0, 0], 0, 8, [0] * 6)
    # a count that cannot be
    for bad in (-1, 71):
        p.count = bad
        p.dev["count"].copy_(_ints([bad]))
        p.check([30, 8, 0, 0, 0, -1], 64, 64, [0] * 6)


def test_plan_loses_pages_that_find_no_room():
    rng = np.random.default_rng(4)
    p = Pool(1, 3, 1, 8, 5, 15, rng)
    p.check([40, 40, 40], 120, 40, [0] * 3)
    p.count = 12                                           # but all fifteen are held
    p.dev["count"].copy_(_ints([12]))
    assert p.check([-1, 0, -1], 0, 1, [0] * 3)[3] == B.BAD_PAGE


@pytest.mark.parametrize("seqs,heads", [(1, 1), (70, 3), (3000, 2)])
def test_plan_without_pages(seqs, heads):
    rng = np.random.default_rng([seqs, 1])
    lens = rng.integers(0, 100, (4, seqs, heads))
    n = rng.integers(-1, 30, seqs)
    first = rng.integers(0, 1000, seqs)
    cache = _bare_cache(4, seqs, heads, 120, lens=_ints(lens))
    st = _status()
    cu = torch.zeros(seqs + 1, dtype=torch.int32, device=DEV)
    cap = int(np.maximum(n, 0).sum()) - 5
    cap = max(cap, 1)
    pos = torch.full((cap,), -9, dtype=torch.int32, device=DEV)
    im = nexus.Image(k=cache.k.to(torch.float8_e4m3fn), v=cache.v.to(torch.float8_e4m3fn),
                     k_scale=torch.ones(4 * seqs * heads * 4, device=DEV),
                     v_scale=torch.ones(4 * seqs * heads * 4, device=DEV),
                     rows=_ints(lens // 32 * 32))
    nexus.plan(cache, None, _ints(n), cu, st, max_tokens=30, token_pos=pos, first_pos=_ints(first),
               image=im)
    torch.cuda.synchronize()
    want_rows = lens // 32 * 32
    want_rows[:, n < 0] = 0
    rcu, _, rpos, _, status = B.plan_plain(lens, n, 120, tokens=cap, max_tokens=30, first_pos=first)
    assert cu.cpu().tolist() == rcu and int(st.item()) == status
    assert pos.cpu().tolist() == rpos + [-9] * (cap - len(rpos))
    assert np.array_equal(cache.lens.cpu().numpy(), lens)
    assert np.array_equal(im.rows.cpu().numpy(), want_rows)


@pytest.mark.parametrize("seqs", [1, 30, 64, 65, 1000, 8192])
@pytest.mark.parametrize("where", ["pos", "seq", "cu"])
def test_plan_first_positions_in_an_array_that_it_writes(seqs, where):
    # first_pos at the front of token_pos, of token_seq or of cu_tokens: all of it is read before
    # anything is written there, also where tokens and sequences are not one to one
    rng = np.random.default_rng([seqs, 2])
    for most in (2, 40):
        n = rng.integers(-1, most, seqs)
        n[0] = 1
        first = rng.integers(0, 1 << 30, seqs)
        lens = rng.integers(0, 50, (2, seqs, 1))
        N = int(np.maximum(n, 0).sum())
        pos, seq = (torch.full((max(N, seqs),), -9, dtype=torch.int32, device=DEV) for _ in range(2))
        cu, st = torch.full((seqs + 1,), -9, dtype=torch.int32, device=DEV), _status()
        at = {"pos": pos, "seq": seq, "cu": cu}[where][:seqs]
        at.copy_(_ints(first))
        cache = _bare_cache(2, seqs, 1, 100, lens=_ints(lens))
        nexus.plan(cache, None, _ints(n), cu, st, max_tokens=most, token_seq=seq, token_pos=pos,
                   first_pos=at)
        torch.cuda.synchronize()
        rcu, rseq, rpos, _, status = B.plan_plain(lens, n, 100, tokens=len(pos), max_tokens=most,
                                                  first_pos=first)
        assert int(st.item()) == status == 0 and cu.cpu().tolist() == rcu
        assert seq[:N].cpu().tolist() == rseq and pos[:N].cpu().tolist() == rpos


def test_plan_largest_prompts():
    # pages by the ten thousands, one sequence with most of the tokens
    rng = np.random.default_rng(9)
    p = Pool(1, 50, 2, 8, 9000, 50 * 700 + 9000, rng)
    n = rng.integers(1, 5000, 50)
    n[17] = 70000
    p.check(n, int(n.sum()), 70000, [0] * 50)
    p.disjoint()
    n[:] = -1
    p.check(n, 0, 1, [0] * 50)
    assert p.count == p.pages


# ---------------------------------------------------------------------------
# verify
# ---------------------------------------------------------------------------

def _probs(rng, N, V, near=None):
    x = rng.standard_normal((N, V)) * 2.5
    if near is not None:
        x = near + 0.6 * rng.standard_normal((N, V))
    e = np.exp(x - x.max(1, keepdims=True))
    return (e / e.sum(1, keepdims=True)).astype(np.float32), x


def _check_verify(n, V, dtype=F32, drafted=True, seed=0, layers=2, kv_heads=3, image=False,
                  page=0, pad=0, q_pad=0, mutate=None, in_place=False, max_tokens=None, spare=0):
    """pad, q_pad: columns between two rows (and before the first) of p and q."""
    rng = np.random.default_rng([seed, V, len(n)])
    S, N = len(n), int(sum(n))
    cu = np.concatenate([[0], np.cumsum(n)]).astype(int)
    p, logits = _probs(rng, N, V)
    q = _probs(rng, N, V, logits)[0] if drafted else None
    src = p if q is None else q
    token = np.zeros(N, np.int64)
    for i in range(N - 1):
        token[i + 1] = np.searchsorted(np.cumsum(src[i].astype(float)),
                                       rng.random() * float(src[i].sum(dtype=float)))
    token = np.clip(token, 0, V - 1)
    u, u_draw = rng.random(N).astype(np.float32), rng.random(S).astype(np.float32)
    u, u_draw = np.minimum(u, np.float32(1 - 2.0 ** -24)), np.minimum(u_draw, np.float32(1 - 2.0 ** -24))
    if mutate:
        mutate(p, q, token, u, u_draw)

    def put(x, pad):
        t = torch.full((N, V + pad), math.nan, dtype=dtype, device=DEV)
        t = t[:, pad // 2:pad // 2 + V] if pad else t
        t.copy_(torch.as_tensor(x).to(dtype))
        return t, t.float().cpu().numpy()

    pd, p = put(p, pad)
    qd, q = put(q, q_pad) if drafted else (None, None)
    lens = rng.integers(max(n), 4000, (layers, S, kv_heads))
    b = min(32, page) if page else 32
    per = -(-4000 // (page or 32))
    cache = _bare_cache(layers, S, kv_heads, per * page if page else 4000, page, 7 if page else 0,
                        _ints(np.zeros((S, per))) if page else None, lens=_ints(lens))
    im = None
    if image:
        blocks = 64 // 64 // b if page else layers * S * kv_heads * 125
        im = nexus.Image(k=cache.k.to(torch.float8_e4m3fn), v=cache.v.to(torch.float8_e4m3fn),
                         k_scale=torch.ones(blocks, device=DEV),
                         v_scale=torch.ones(blocks, device=DEV), rows=_ints(lens // b * b))
    st = _status()
    out = torch.full((N + spare,), -9, dtype=torch.int32, device=DEV)
    emitted = torch.full((S,), -9, dtype=torch.int32, device=DEV)
    uniform = len(set(n)) == 1 and not spare
    lens_in = None if in_place else cache.lens.clone()
    if lens_in is not None:
        cache.lens.fill_(-5)
    nexus.verify(cache, _ints(token), pd, torch.as_tensor(u, device=DEV),
                 torch.as_tensor(u_draw, device=DEV), out[:N], emitted, st,
                 max_tokens=max_tokens or max(max(n), 1), cu_tokens=None if uniform else _ints(cu), q=qd,
                 lens_in=lens_in, image=im)
    torch.cuda.synchronize()
    assert nexus.last_launch_names() == ["verify"]
    ro, re, gone, status = B.verify_plain(token, p, q, u, u_draw, cu)
    assert int(st.item()) == status
    assert out.cpu().tolist() == ro + [-9] * spare and emitted.cpu().tolist() == re
    want = lens - np.array(gone)[None, :, None]
    assert np.array_equal(cache.lens.cpu().numpy(), want)
    if image:
        rows = np.minimum(lens // b * b, (lens - np.array(gone)[None, :, None]) // b * b)
        assert np.array_equal(im.rows.cpu().numpy(), rows)
    return re


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("V", [1, 2, 3, 5, 31, 127, 128, 129, 511, 2047, 2048, 2049, 4097, 8191,
                               16385, 50257])
def test_verify_every_vocabulary(V, drafted, dtype):
    _check_verify([3, 1, 0, 5, 2], V, dtype, drafted, seed=V)


@pytest.mark.parametrize("drafted", [True, False])
def test_verify_largest_vocabularies(drafted):
    _check_verify([2, 4], 131072, drafted=drafted)
    _check_verify([2], (1 << 20) - 1, drafted=drafted)
    _check_verify([2], 1 << 20, BF, drafted=drafted)


@pytest.mark.parametrize("seqs", [1, 2, 37, 38, 39, 75, 77, 151, 153, 303, 305, 700])
def test_verify_every_number_of_sequences(seqs):
    rng = np.random.default_rng(seqs)
    n = list(rng.integers(0, 5, seqs))
    n[0] = 4
    kept = _check_verify(n, 9001, seed=seqs, layers=1, kv_heads=2)
    assert seqs < 50 or len(set(kept)) >= 4


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("pad,q_pad", [(1, 1), (2, 2), (3, 1), (5, 0), (0, 7), (4, 2), (6, 6)])
def test_verify_rows_at_any_distance(pad, q_pad, dtype):
    _check_verify([4, 3, 4], 3001, dtype, pad=pad, q_pad=q_pad, seed=pad)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("page", [0, 8, 16, 64])
def test_verify_takes_rows_back(page, in_place):
    _check_verify([6, 2, 0, 9], 300, page=page, image=page == 0, layers=5, in_place=in_place)


def test_verify_many_drafts():
    # more drafts than a thread block has threads, all kept but one
    def keep(p, q, token, u, u_draw):
        u[:] = 0
        u[1100] = 1 - 2.0 ** -24
        q[1100, token[1101]] = 1.0
    got = _check_verify([1300, 700], 40, mutate=keep)
    assert got == [1101, 700]


def test_verify_uniform_ends_and_odd_values():
    def edges(p, q, token, u, u_draw):
        u[:], u_draw[:] = 0, 0
        u[4:] = np.float32(1 - 2.0 ** -24)
        u_draw[1:] = np.float32(1 - 2.0 ** -24)
    for V in (7, 5000):
        _check_verify([4, 4, 4], V, mutate=edges)

    def outside(p, q, token, u, u_draw):
        u[0], u[2], u[3] = math.nan, -3.0, 2.0
        u_draw[:] = [-1.0, 1.0, math.nan]
    _check_verify([4, 4, 4], 1000, mutate=outside)

    def odd(p, q, token, u, u_draw):
        p[:, 1], p[:, 2], p[:, 3] = math.nan, -0.5, math.inf
        q[:, 4], q[:, 5] = math.nan, math.inf
        token[2], token[3], token[5] = 1, 2, 4
    _check_verify([4, 4, 4], 900, mutate=odd)


def test_verify_nothing_left_and_nothing_at_all():
    def same(p, q, token, u, u_draw):
        # rejected although p = q: u q < p fails only for u = 1, so p is a little less everywhere
        q[:] = p * np.float32(1.5)
        u[:] = np.float32(1 - 2.0 ** -24)
    _check_verify([3, 3], 700, mutate=same)          # p - q is nowhere positive: p itself

    def zero(p, q, token, u, u_draw):
        p[:] = 0
        u[:] = 0.5
    _check_verify([3, 1], 5000, mutate=zero)         # NX_DEV_BAD_PROBS

    def one(p, q, token, u, u_draw):
        p[:] = 0
        p[:, 4999] = 2.0 ** -42                      # the smallest weight that counts
        p[:, 17] = 2.0 ** -43
        u[:] = 0.5
    _check_verify([1, 1], 5000, mutate=one, drafted=False)


@pytest.mark.parametrize("V", [7, 700, 9001])
def test_verify_weights_below_the_smallest_count_as_none(V):
    # 2^-43 (1 + 2^-23 at most) is no weight, however many columns have it
    def below(p, q, token, u, u_draw):
        p[:], q[:] = 2.0 ** -43, 0
        u[:] = np.float32(1 - 2.0 ** -24)
        p[0] = np.nextafter(np.float32(2.0 ** -42), np.float32(0))
    for n in ([1, 1], [3, 2]):
        kept = _check_verify(n, V, mutate=below)         # NX_DEV_BAD_PROBS, token 0
        assert kept == n                                 # (the drafts' q is 0: they stay)

    # as what is left of p behind q: p itself is drawn from, columns that q excludes among them
    def left(p, q, token, u, u_draw):
        p[:] = 0
        p[:, 0], p[:, 1] = 0.75, 0.25
        q[:] = p
        p[:, 2:] = 2.0 ** -43
        u[:] = np.float32(1 - 2.0 ** -24)
        q[:, 0], q[:, 1] = 0.875, 0.5
        token[:] = 0
        u_draw[:] = [0.25, 0.875]
    assert _check_verify([3, 3], V, mutate=left) == [1, 1]


@pytest.mark.parametrize("drafted", [True, False])
def test_verify_drafts_outside_the_vocabulary(drafted):
    def bad(p, q, token, u, u_draw):
        u[:] = 0
        token[2], token[5] = 1000, -1
    assert _check_verify([4, 4], 1000, drafted=drafted, mutate=bad) == [2, 1]


@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("far", [1000, 1001, 1003, 2 ** 31 - 1, -2 ** 31])
def test_verify_first_draft_outside_draws_from_the_whole_row(far, drafted):
    def bad(p, q, token, u, u_draw):
        u[:] = 0
        token[1] = far
    assert _check_verify([3, 1], 1000, drafted=drafted, mutate=bad) == [1, 1]


def test_verify_faults_are_flagged():
    cache = _bare_cache(1, 3, 2, 50, lens=_ints([[[5, 1], [51, 5], [-1, 7]]]))
    token, out = _ints([0, 1, 1] * 3), torch.full((9,), -9, dtype=torch.int32, device=DEV)
    p = torch.zeros(9, 4, device=DEV)
    p[:, 0] = 1                                      # draft 1 always goes: two rows back
    u, ud, em = torch.full((9,), 0.5, device=DEV), torch.zeros(3, device=DEV), _ints([-9] * 3)
    st = _status()
    nexus.verify(cache, token, p, u, ud, out, em, st, max_tokens=3)
    torch.cuda.synchronize()
    assert int(st.item()) == nexus.NX_DEV_BAD_LEN
    assert cache.lens.cpu().tolist() == [[[3, 1], [51, 3], [-1, 5]]]
    assert out.cpu().tolist() == [0, -1, -1] * 3 and em.cpu().tolist() == [1, 1, 1]
    # a sequence whose tokens are not where they should be is left out
    st.zero_()
    out.fill_(-9)
    nexus.verify(cache, token, p, u, ud, out, em, st, max_tokens=3, cu_tokens=_ints([0, 3, 1, 9]))
    torch.cuda.synchronize()
    assert int(st.item()) == nexus.NX_DEV_BAD_TOKENS | nexus.NX_DEV_BAD_LEN
    assert em.cpu().tolist() == [1, 0, 0] and out.cpu().tolist() == [0, -1, -1] + [-9] * 6


def test_verify_padded_batch_and_none():
    _check_verify([2, 0, 3], 500, spare=4, max_tokens=7)
    cache = _bare_cache(1, 2, 1, 50, lens=_ints([[[5], [6]]]))
    em, st, none = _ints([7, 7]), _status(), _ints([])
    nexus.verify(cache, none, torch.zeros(0, 8, device=DEV), torch.zeros(0, device=DEV),
                 torch.zeros(2, device=DEV), none, em, st, max_tokens=1, cu_tokens=_ints([0, 0, 0]))
    torch.cuda.synchronize()
    assert em.cpu().tolist() == [0, 0] and cache.lens.cpu().tolist() == [[[5], [6]]]


@pytest.mark.parametrize("V", [1025, 2049, 4100, 8193])
def test_verify_blocks_of_a_sequence_that_start_apart(V):
    # few columns to each of a sequence's two to eight thread blocks, next to another stream that keeps
    # the GPU's places taken: a block may be done with its sum long before the others have begun, and
    # must not send it to them until they have
    rng = np.random.default_rng(V)
    S, calls = 40, 60
    p, _ = _probs(rng, S, V)
    u_draw = np.minimum(rng.random(S).astype(np.float32), np.float32(1 - 2.0 ** -24))
    want = B.verify_plain([0] * S, p, None, np.zeros(S), u_draw, list(range(S + 1)))
    cache = _bare_cache(1, S, 1, 8, lens=torch.full((1, S, 1), 4, dtype=torch.int32, device=DEV))
    pd, ud, u = torch.as_tensor(p, device=DEV), torch.as_tensor(u_draw, device=DEV), torch.zeros(S, device=DEV)
    token, st = _ints([0] * S), _status()
    out, em = torch.full((calls, S), -9, dtype=torch.int32, device=DEV), _ints([-9] * S)
    busy = torch.zeros(1 << 22, device=DEV)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(calls):
        with torch.cuda.stream(other):
            busy.add_(1.0)
        nexus.verify(cache, token, pd, u, ud, out[i], em, st, max_tokens=1)
    torch.cuda.synchronize()
    assert int(st.item()) == want[3] == 0 and em.cpu().tolist() == want[1]
    assert out.cpu().tolist() == [want[0]] * calls


def test_verify_gives_the_models_distribution():
    # 60000 sequences with the same p and q, drafts drawn from q: the first token is distributed
    # like p. Five standard deviations of a count out of n: 5 sqrt(n p (1 - p)), missed by chance
    # once in 10^6 per column
    n, V = 60000, 6
    p = torch.tensor([0.05, 0.3, 0.15, 0.2, 0.3, 0.0], device=DEV)
    q = torch.tensor([0.3, 0.1, 0.15, 0.25, 0.1, 0.1], device=DEV)
    g = torch.Generator(device=DEV).manual_seed(5)
    draft = torch.multinomial(q, n, replacement=True, generator=g).int()
    token = torch.stack([torch.zeros_like(draft), draft], 1).reshape(-1).contiguous()
    cache = _bare_cache(1, n, 1, 8, lens=torch.full((1, n, 1), 4, dtype=torch.int32, device=DEV))
    out, em = torch.empty_like(token), torch.empty(n, dtype=torch.int32, device=DEV)
    st = _status()
    nexus.verify(cache, token, p.expand(2 * n, V), torch.rand(2 * n, device=DEV, generator=g),
                 torch.rand(n, device=DEV, generator=g), out, em, st, max_tokens=2,
                 q=q.expand(2 * n, V))
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    count = torch.bincount(out.view(n, 2)[:, 0].long(), minlength=V).double().cpu()
    want = p.double().cpu() * n
    assert torch.all((count - want).abs() <= 5 * (want * (1 - want / n)).sqrt() + 1e-9), count
    kept = float((em == 2).sum())
    overlap = float(torch.minimum(p, q).sum()) * n
    assert abs(kept - overlap) <= 5 * math.sqrt(overlap * (1 - overlap / n))


# ---------------------------------------------------------------------------
# attend_shared
# ---------------------------------------------------------------------------

def _image(cache):
    im = nexus.new_image(cache)
    im.k.view(torch.uint8).fill_(0x7F)                               # NaN
    im.v.view(torch.uint8).fill_(0x7F)
    im.k_scale.fill_(math.nan)
    im.v_scale.fill_(math.nan)
    return im


def _rows(c, im, layer, s, h):
    """Keys and values that a slice holds, in float64, from the image where it holds them."""
    T = int(c.lens[layer, s, h])
    got = []
    for name in ("k", "v"):
        x = getattr(c, name)[c.at(layer, s, h, T)].double()
        if im is not None:
            r = int(im["rows"][layer, s, h])
            at = c.at(layer, s, h, r)
            j = torch.arange(r)
            scale = im[name + "_scale"][layer, c.table[s].long()[j // c.page], h, j % c.page // c.b] \
                if c.page else im[name + "_scale"][layer, s, h, j // c.b]
            x[:r] = im[name][at].double() * scale.double()[:, None]
        got.append(x)
    return got


def _check_shared(own, pre, groups, n, layer=0, causal=True, image=False, pre_image=False,
                  scale=None, uniform=False, max_shared=None, mutate=None, want_status=0,
                  refs=True, spare=0):
    """own, pre: Case. groups: cu_seqs (None: one prefix for all)."""
    HG, N, d = own.H * own.G, int(sum(n)), own.d
    q = torch.randn(N + spare, HG + 3, d, generator=own.g).to(own.dtype)
    if mutate:
        mutate(own, pre, q)
    cache, prefix, st = own.device_cache(), pre.device_cache(), _status()
    ims = []
    for flag, c in ((image, cache), (pre_image, prefix)):
        ims.append(None)
        if flag:
            ims[-1] = _image(c)
            nexus.quantize(c, ims[-1], st)
    qd = q.to(DEV)[:, 1:1 + HG]                                      # a strided view
    out = torch.full((N + spare, HG + 2, d), math.nan, dtype=own.dtype, device=DEV)[:, 1:-1]
    lse = torch.full((N + spare, HG), math.nan, device=DEV)
    cu = np.concatenate([[0], np.cumsum(n)]).astype(int)
    cu_seqs = [0, own.S] if groups is None else list(groups)
    most = max([1] + [int(cu[b] - cu[a]) for a, b in zip(cu_seqs, cu_seqs[1:])
                      if 0 <= a <= b <= own.S])
    mt = max(max(n), 1)
    kw = dict(prefix=prefix, max_tokens=mt, max_shared=max_shared or most,
              cu_seqs=None if groups is None else _ints(groups),
              cu_tokens=None if uniform else _ints(cu), causal=causal, scale=scale, image=ims[0],
              prefix_image=ims[1])
    ws = nexus.alloc_attend_shared_workspace(cache, prefix, tokens=N + spare, max_tokens=mt,
                                             max_shared=kw["max_shared"])
    ws.fill_(0xFF)                                                   # it may hold anything
    torch.cuda.synchronize()
    nexus.attend_shared(cache, layer, qd, out, ws, st, lse=lse, **kw)
    names = nexus.last_launch_names()
    out2 = torch.full((N + spare, HG, d), math.nan, dtype=own.dtype, device=DEV)
    nexus.attend_shared(cache, layer, qd, out2, ws, st, **kw)        # no lse, used workspace
    torch.cuda.synchronize()
    assert int(st.item()) == want_status
    bits = torch.int16 if own.dtype == BF else torch.int32           # (NaN too)
    assert torch.equal(out2[:N].view(bits), out[:N].contiguous().view(bits))   # the same each time
    assert torch.all(out2[N:].isnan()) and torch.all(lse[N:].isnan())
    if not refs:
        return out, lse, names
    sc = d ** -0.5 if scale is None else scale
    host = [None if im is None else dict(k=im.k.float().cpu(), v=im.v.float().cpu(),
                                         k_scale=im.k_scale.cpu(), v_scale=im.v_scale.cpu(),
                                         rows=im.rows.cpu()) for im in ims]
    for s, m in enumerate(n):
        a = cu[s]
        p = B.prefix_of(cu_seqs, s)
        for h in range(own.H):
            T = int(own.lens[layer, s, h])
            k, v = _rows(own, host[0], layer, s, h)
            M = [(T - (m - 1 - i) if causal else T) for i in range(m) for _ in range(own.G)]
            parts = [(k, v, M)]
            before = 0
            if p >= 0:
                k, v = _rows(pre, host[1], layer, p, h)
                before = k.shape[0]
                parts.insert(0, (k, v, [before] * len(M)))
            rows = q[a:a + m, 1 + h * own.G:1 + (h + 1) * own.G].reshape(-1, d)
            ro, rl, A, big = B.shared64(rows, parts, sc)
            got = out[a:a + m, h * own.G:(h + 1) * own.G].reshape(-1, d).cpu().double()
            gl = lse[a:a + m, h * own.G:(h + 1) * own.G].reshape(-1).cpu().double()
            dx = abs(sc) * big * (2.0 ** -24 * (d + 8) if own.dtype == BF else 2.0 ** -20)
            w = (2.0 ** -8 if own.dtype == BF else 2.0 ** -19) + 2.0 ** -20
            tol = HALF[own.dtype] * ro.abs() + (w + 2 * dx)[:, None] * A + 1e-30
            err = (got - ro).abs()
            assert torch.all(err <= tol), (s, h, float((err / tol).max()))
            none = torch.tensor([before + max(0, x) <= 0 for x in M], dtype=torch.bool)
            assert torch.all(torch.isneginf(gl[none])) and torch.all(got[none] == 0)
            el = (gl - rl).abs()[~none]
            assert torch.all(el <= (dx + 2.0 ** -18 * (1 + rl.abs()))[~none]), (s, h)
    return out, lse, names


KINDS = {"bf16": dict(), "bf16_64": dict(d=64), "f32": dict(dtype=F32), "f32_64": dict(dtype=F32, d=64)}


def _pair(kind, seqs, prefixes, lens, pre_lens, page=0, pre_page=None, **kw):
    kw = {**dict(kv_heads=2, group=4), **KINDS[kind], **kw}
    pre_page = page if pre_page is None else pre_page
    own = Case(seqs=seqs, page=page, capacity=max(8, int(np.max(lens))), lens=lens, seed=1, **kw)
    pre = Case(seqs=prefixes, page=pre_page, capacity=max(8, int(np.max(pre_lens))), lens=pre_lens,
               seed=2, **kw)
    return own, pre


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("rows", [0, 1, 15, 64, 65, 300, 2500])
def test_shared_one_token_every_prefix_length(kind, rows):
    own, pre = _pair(kind, 5, 1, [[1, 7], [16, 33], [64, 65], [100, 1], [300, 2]],
                     [[rows, max(0, rows - 3)]])
    _check_shared(own, pre, None, [1] * 5, uniform=True)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("seqs,tokens", [(2, 1), (4, 1), (5, 1), (9, 2), (17, 2), (33, 1), (70, 1), (4, 40),
                                         (3, 130)])
def test_shared_query_rows(kind, causal, seqs, tokens):
    # 8 to 1560 query rows behind a prefix: every kernel, and several row tiles of one
    rng = np.random.default_rng([seqs, tokens])
    own, pre = _pair(kind, seqs, 1, rng.integers(tokens, tokens + 90, (seqs, 2)), [[333, 170]])
    _check_shared(own, pre, None, [tokens] * seqs, causal=causal)


@pytest.mark.parametrize("image", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("each", [5, 20, 40])
@pytest.mark.parametrize("lens", [[[4200, 4096]], [[4500, 0], [1, 4200], [64, 4097]]], ids=["one", "three"])
def test_shared_prefixes_on_the_tensor_cores(lens, each, d, image):
    # 20, 80 and 160 query rows to a prefix, whole shares of blocks for units of any length
    P = len(lens)
    rng = np.random.default_rng(each)
    own, pre = _pair("bf16", P * each, P, rng.integers(1, 40, (P * each, 2)), lens, d=d, page=16)
    groups = [each * i for i in range(P + 1)]
    _, _, names = _check_shared(own, pre, groups, [1] * (P * each), pre_image=image)
    assert names[0] == "attend_tc" and names[-1] == "attend_meet"


@pytest.mark.parametrize("image,slots", [(False, 1030), (True, 1930)])
@pytest.mark.parametrize("d", [64, 128])
def test_shared_pieces_of_one_tile(d, image, slots):
    # up to 128 query rows, so that a row tile's slots are dealt to two streams, and 17 or 31 tiles (of 64
    # slots) to each unit in shares of 2 or 3: in a piece of one the second stream has none, and its warp
    # nothing to wait for between the block's share and the first piece's results. The same bits again
    # and again.
    own, pre = _pair("bf16", 32, 1, 5, [[slots] * 8], d=d, kv_heads=8)
    first, _, names = _check_shared(own, pre, None, [1] * 32, pre_image=image)
    assert names[0] == "attend_tc" and names[-1] == "attend_meet"
    own, pre = _pair("bf16", 32, 1, 5, [[slots] * 8], d=d, kv_heads=8)
    cache, prefix, st = own.device_cache(), pre.device_cache(), _status()
    im = None
    if image:
        im = _image(prefix)
        nexus.quantize(prefix, im, st)
    q = torch.randn(32, 32 + 3, d, generator=own.g).to(own.dtype).to(DEV)[:, 1:33]
    ws = nexus.alloc_attend_shared_workspace(cache, prefix, tokens=32, max_tokens=1, max_shared=32)
    out = torch.full((100, 32, 32, d), math.nan, dtype=BF, device=DEV)
    for i in range(100):
        nexus.attend_shared(cache, 0, q, out[i], ws, st, prefix=prefix, max_tokens=1, max_shared=32,
                            prefix_image=im)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and torch.all(out == first[None])


@pytest.mark.parametrize("prefixes,rows", [(5, 200), (9, 20)])
def test_shared_many_prefix_units(prefixes, rows):
    # 40 and 72 units of the tensor cores, next to so many own rows that the 40 get 38 blocks: shares
    # that go on from one unit to the next
    each = 80
    rng = np.random.default_rng(prefixes)
    own, pre = _pair("bf16_64", prefixes * each, prefixes,
                     rng.integers(rows // 2, rows * 3 // 2, (prefixes * each, 4)),
                     rng.integers(900, 1000, (prefixes, 4)), kv_heads=4)
    groups = [each * i for i in range(prefixes + 1)]
    _, _, names = _check_shared(own, pre, groups, [1] * (prefixes * each))
    assert names[0] == "attend_tc" and names[-1] == "attend_meet"


@pytest.mark.parametrize("kind,image", [("bf16", False), ("bf16", True), ("f32", False)])
@pytest.mark.parametrize("rows", [40, 4200])
def test_shared_long_own_slices(rows, kind, image):
    # own slices so long that their tiles are shared evenly and joined, in either order of the passes
    rng = np.random.default_rng(rows)
    own, pre = _pair(kind, 20, 1, rng.integers(4000, 9000, (20, 2)), [[rows, rows - 7]])
    _, _, names = _check_shared(own, pre, None, [1] * 20, image=image)
    assert "attend_join" in names and ("attend_meet" in names) == (rows == 4200 and kind == "bf16")


def test_shared_prefixes_that_nobody_shares():
    own, pre = _pair("bf16", 6, 2, 30, [[4200, 4000], [4100, 4200]])
    a, _, names = _check_shared(own, pre, [3, 3, 3], [1] * 6, max_shared=40)
    assert names[0] == "attend_tc" and names[-1] == "attend_meet"


@pytest.mark.parametrize("image", ["none", "own", "both"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [20, 900])
def test_shared_chunks_of_long_slices(rows, d, image):
    # own slices with many query rows, behind a prefix of few rows and of many: both of its parts by
    # either kernel
    own, pre = _pair("bf16", 3, 1, [[1400, 1201], [1399, 96], [1100, 1340]], [[rows, rows - 5]], d=d,
                     page=16)
    _, _, names = _check_shared(own, pre, None, [96, 95, 60], image=image != "none",
                                pre_image=image == "both")
    assert "attend_tc_join" in names and ("attend_meet" in names) == (rows == 900)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("page,pre_page", [(8, 8), (16, 0), (0, 16), (32, 64), (128, 128)])
def test_shared_several_prefixes_ragged_and_paged(kind, page, pre_page):
    rng = np.random.default_rng(page)
    n = rng.integers(0, 6, 23)
    n[4] = 5
    own, pre = _pair(kind, 23, 6, rng.integers(5, 200, (23, 2)), rng.integers(0, 500, (6, 2)),
                     page=page, pre_page=pre_page)
    # sequences 0 and 1 have no prefix, nor has the last; prefixes of one and of no sequence
    _check_shared(own, pre, [2, 9, 9, 10, 17, 17, 22], list(n))


@pytest.mark.parametrize("which", ["own", "prefix", "both"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [0, 8, 32])
@pytest.mark.parametrize("seqs,tokens", [(1, 1), (3, 2), (12, 1), (30, 2)])
def test_shared_images(which, d, page, seqs, tokens):
    rng = np.random.default_rng([d, page, seqs])
    own, pre = _pair("bf16", seqs, 1, rng.integers(tokens, 150, (seqs, 2)), [[290, 77]], page=page,
                     d=d)
    _check_shared(own, pre, None, [tokens] * seqs, image=which != "prefix",
                  pre_image=which != "own")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("seqs", [3, 20, 100])
def test_shared_long_prefix_split_over_blocks(kind, seqs):
    rng = np.random.default_rng(seqs)
    own, pre = _pair(kind, seqs, 1, rng.integers(1, 60, (seqs, 2)), [[20000, 17001]], page=16)
    out, _, names = _check_shared(own, pre, None, [1] * seqs)
    assert names[-1].startswith("attend") and len(names) >= 2


def test_shared_tokens_that_see_nothing_of_their_own():
    # slices with fewer rows than tokens: the first tokens see the prefix only, or nothing at all
    own, pre = _pair("bf16", 3, 1, [[2, 0], [0, 5], [1, 1]], [[40, 0]])
    _check_shared(own, pre, [0, 2], [4, 5, 3])
    own, pre = _pair("f32", 3, 1, [[2, 0], [0, 5], [1, 1]], [[40, 0]])
    _check_shared(own, pre, [1, 3], [4, 5, 3])


def test_shared_layers_scales_and_padding():
    own, pre = _pair("bf16", 4, 2, 50, 70, layers=3)
    _check_shared(own, pre, [0, 2, 4], [1, 2, 0, 1], layer=2, spare=3)
    _check_shared(own, pre, [0, 1, 4], [1, 2, 0, 1], layer=1, scale=0.0)
    _check_shared(own, pre, [0, 3, 4], [1, 1, 1, 1], scale=-0.3, max_shared=100)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("far", ["prefix", "own"])
def test_shared_parts_far_apart(kind, far):
    # one part's logits hundreds above the other's
    def mutate(own, pre, q):
        for c, x in ((pre, 20.0 if far == "prefix" else -20.0), (own, -20.0 if far == "prefix" else 20.0)):
            for s in range(c.S):
                for h in range(c.H):
                    at = c.at(0, s, h, int(c.lens[0, s, h]))
                    rows = c.k[at]
                    rows[:, 0] = x
                    c.k[at] = rows
        q[..., 0] = 30.0
    for seqs in (2, 40):
        own, pre = _pair(kind, seqs, 1, 30, 90)
        _check_shared(own, pre, None, [1] * seqs, mutate=mutate)


@pytest.mark.parametrize("seqs", [2, 6, 40])
def test_shared_rows_that_are_not_finite_reach_their_own_tokens_only(seqs):
    own, pre = _pair("bf16", 2 * seqs, 2, 60, 100)
    clean = _check_shared(own, pre, [0, seqs, 2 * seqs], [1] * 2 * seqs)[0]
    own, pre = _pair("bf16", 2 * seqs, 2, 60, 100)

    def mutate(own, pre, q):
        pre.v[pre.at(0, 1, 0, 6, 5)] = math.inf                      # prefix 1, head 0
        own.v[own.at(0, 0, 1, 8, 7)] = math.nan                      # sequence 0, head 1
    out, _, _ = _check_shared(own, pre, [0, seqs, 2 * seqs], [1] * 2 * seqs, mutate=mutate,
                              refs=False)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[seqs:, :4] = True
    bad[0, 4:] = True
    assert torch.all(~torch.isfinite(out[bad])) and torch.equal(out[~bad], clean[~bad])


def test_shared_prefix_like_a_whole_cache():
    # the same rows as one cache: attend over prefix and own rows behind one another
    own, pre = _pair("bf16", 3, 1, 40, 500, kv_heads=2)
    out, lse, _ = _check_shared(own, pre, None, [2, 2, 2])
    whole = Case(seqs=3, kv_heads=2, group=4, capacity=540, lens=540)
    for s in range(3):
        for h in range(2):
            for t, o, p in ((whole.k, own.k, pre.k), (whole.v, own.v, pre.v)):
                t[0, s, h, :500], t[0, s, h, 500:] = p[0, 0, h, :500], o[0, s, h, :40]
    cache, st = whole.device_cache(), _status()
    ws = nexus.alloc_attend_workspace(cache, tokens=6, max_tokens=2)
    q = torch.randn(6, 8, 128, generator=own.g).to(DEV, BF)
    a = torch.empty(6, 8, 128, dtype=BF, device=DEV)
    b = torch.empty_like(a)
    la, lb = torch.empty(6, 8, device=DEV), torch.empty(6, 8, device=DEV)
    nexus.attend(cache, 0, q, a, ws, st, max_tokens=2, lse=la)
    c, p = own.device_cache(), pre.device_cache()
    ws = nexus.alloc_attend_shared_workspace(c, p, tokens=6, max_tokens=2, max_shared=6)
    nexus.attend_shared(c, 0, q, b, ws, st, prefix=p, max_tokens=2, max_shared=6, lse=lb)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    # both are within a rounding to bf16 and 2^-8 of sum p |v| (at most max |v|, below 6) of the
    # same numbers
    assert float((a.float() - b.float()).abs().max()) <= 4 * 2.0 ** -8 * 6
    assert float((la - lb).abs().max()) <= 2.0 ** -16 * float(la.abs().max())


def test_shared_faults_are_flagged():
    n = [2, 3, 2, 1]
    # (60 rows: every unit is one thread block's, so that equal sums are equal bits)
    own, pre = _pair("bf16", 4, 2, 40, 60, page=16)
    good, _, _ = _check_shared(own, pre, [0, 2, 4], n)

    def again(**kw):
        own, pre = _pair("bf16", 4, 2, 40, 60, page=16)
        groups = kw.pop("groups", [0, 2, 4])
        return _check_shared(own, pre, groups, kw.pop("n", n), refs=False, **kw)[0]

    own, pre = _pair("bf16", 4, 2, 40, 60, page=16)
    alone, _, _ = _check_shared(own, pre, [0, 0, 0], n)              # nobody has a prefix
    # boundaries that make no sense: those prefixes count as empty
    out = again(groups=[0, 2, 5], want_status=nexus.NX_DEV_BAD_TOKENS)
    assert torch.equal(out[:5], good[:5]) and torch.equal(out[5:], alone[5:])
    out = again(groups=[3, 2, 4], max_shared=5, want_status=nexus.NX_DEV_BAD_TOKENS)
    assert torch.equal(out[:5], alone[:5]) and torch.equal(out[5:], good[5:])
    out = again(groups=[-1, 2, 4], max_shared=5, want_status=nexus.NX_DEV_BAD_TOKENS)
    assert torch.equal(out[:5], alone[:5]) and torch.equal(out[5:], good[5:])
    # more tokens than max_shared allows
    out = again(max_shared=4, want_status=nexus.NX_DEV_BAD_TOKENS)
    assert torch.equal(out[:5], alone[:5]) and torch.equal(out[5:], good[5:])

    # a prefix with a bad length counts as empty, a bad page's rows are left out
    def bad_len(own, pre, q):
        pre.lens[0, 1, 0] = pre.capacity + 1
    own, pre = _pair("bf16", 4, 2, 40, 60, page=16)
    out = _check_shared(own, pre, [0, 2, 4], n, mutate=bad_len, refs=False,
                        want_status=nexus.NX_DEV_BAD_LEN)[0]
    assert torch.equal(out[:5], good[:5]) and torch.equal(out[5:, 4:], good[5:, 4:])
    assert torch.equal(out[5:, :4], alone[5:, :4])

    def bad_page(own, pre, q):
        pre.table[0, 2:] = -1
    own, pre = _pair("bf16", 4, 2, 40, 60, page=16)
    out = _check_shared(own, pre, [0, 2, 4], n, mutate=bad_page, refs=False,
                        want_status=nexus.NX_DEV_BAD_PAGE)[0]
    short, prefix = _pair("bf16", 4, 2, 40, 60, page=16)
    prefix.lens[0, 0] = 32
    want = _check_shared(short, prefix, [0, 2, 4], n)[0]
    assert torch.equal(out, want)


def test_shared_sequence_without_its_tokens():
    # a sequence whose tokens are flagged has no output; the others have theirs
    own, pre = _pair("bf16", 3, 1, 40, 60)
    cache, prefix, st = own.device_cache(), pre.device_cache(), _status()
    q = torch.randn(6, 8, 128, generator=own.g).to(DEV, BF)
    out = torch.full_like(q, math.nan)
    ws = nexus.alloc_attend_shared_workspace(cache, prefix, tokens=6, max_tokens=2, max_shared=6)
    nexus.attend_shared(cache, 0, q, out, ws, st, prefix=prefix, max_tokens=2, max_shared=6,
                        cu_tokens=_ints([0, 2, 5, 6]))
    torch.cuda.synchronize()
    assert int(st.item()) == nexus.NX_DEV_BAD_TOKENS                 # three of at most two
    assert torch.all(torch.isfinite(out[:2])) and torch.all(torch.isfinite(out[5]))
    assert torch.all(out[2:5].isnan())


@pytest.mark.parametrize("rows", [60, 5000])
@pytest.mark.parametrize("cu,groups,most,good", [
    ([0, 9, 3, 6], None, 3, [2]),                      # 0: beyond the tokens, 1: decreases
    ([0, 2, 5, 6], None, 2, [0, 2]),                   # 1: three of at most two
    ([0, 2, 6, 3, 6], None, 3, [0, 3]),                # 1: four of at most three, 2: decreases
    ([0, 40, -5, 1, 3, 9, 4, 6], [0, 3, 7], 2, [3, 6]),
])
def test_shared_tokens_of_sequences_that_are_not_flagged(cu, groups, most, good, rows):
    # entries of cu_tokens that make no sense leave out the sequences that they bound; the others have
    # their outputs, whichever kernels take the prefix
    seqs = len(cu) - 1
    own, pre = _pair("bf16", seqs, 2 if groups else 1, 40, [[rows, rows - 3]] * (2 if groups else 1))
    cache, prefix, st = own.device_cache(), pre.device_cache(), _status()
    q = torch.randn(6, 8, 128, generator=own.g).to(BF)
    out = torch.full((6, 8, 128), math.nan, dtype=BF, device=DEV)
    lse = torch.full((6, 8), math.nan, device=DEV)
    ws = nexus.alloc_attend_shared_workspace(cache, prefix, tokens=6, max_tokens=most, max_shared=6)
    ws.fill_(0xFF)
    nexus.attend_shared(cache, 0, q.to(DEV), out, ws, st, prefix=prefix, max_tokens=most, max_shared=6,
                        cu_tokens=_ints(cu), cu_seqs=_ints(groups) if groups else None, lse=lse)
    torch.cuda.synchronize()
    assert ("attend_meet" in nexus.last_launch_names()) == (rows == 5000)
    assert int(st.item()) == nexus.NX_DEV_BAD_TOKENS
    bounds = groups or [0, seqs]
    rest = torch.ones(6, dtype=torch.bool)
    for s in good:
        p, a, b = B.prefix_of(bounds, s), cu[s], cu[s + 1]
        rest[a:b] = False
        for h in range(own.H):
            M = [40 - (b - a - 1 - i) for i in range(b - a) for _ in range(own.G)]
            k, v = _rows(pre, None, 0, p, h)
            parts = [(k, v, [k.shape[0]] * len(M)), (*_rows(own, None, 0, s, h), M)]
            x = q[a:b, h * own.G:(h + 1) * own.G].reshape(-1, 128)
            ro, rl, A, big = B.shared64(x, parts, 128 ** -0.5)
            got = out[a:b, h * own.G:(h + 1) * own.G].reshape(-1, 128).cpu().double()
            gl = lse[a:b, h * own.G:(h + 1) * own.G].reshape(-1).cpu().double()
            dx = 128 ** -0.5 * big * 2.0 ** -24 * 136
            tol = HALF[BF] * ro.abs() + (2.0 ** -8 + 2.0 ** -20 + 2 * dx)[:, None] * A
            assert torch.all((got - ro).abs() <= tol), (s, h)
            assert torch.all((gl - rl).abs() <= dx + 2.0 ** -18 * (1 + rl.abs())), (s, h)
    assert torch.all(out[rest].isnan()) and torch.all(lse[rest].isnan())


# ---------------------------------------------------------------------------
# streams, graphs, and all of them together
# ---------------------------------------------------------------------------

class Server:
    """Sequences behind shared prompts in one pool, with drafts: plan, append, attend_shared,
    verify. The keys of a token are a fixed function of its number and position, so that what a
    sequence should see can be computed from its tokens alone."""

    def __init__(self, seqs=5, layers=2, heads=2, group=2, page=8, per=12, V=50, seed=0):
        self.S, self.L, self.H, self.G, self.d, self.V, self.page = seqs, layers, heads, group, 64, V, page
        g = torch.Generator().manual_seed(seed)
        pages = 2 * 8 + seqs * per
        shape = (layers, pages, heads, page)
        dev = dict(device=DEV)
        self.k, self.v = (torch.zeros(*shape, 64, dtype=BF, **dev) for _ in range(2))
        self.pos = torch.zeros(shape, dtype=torch.int32, **dev)
        self.embed = torch.randn(layers, V, (group * heads + 2 * heads), 64, generator=g).to(BF)
        self.freqs = [10000.0 ** (-2.0 * i / 64) for i in range(32)]
        self.rotary = nexus.Rotary(self.freqs, device=DEV)
        common = dict(k=self.k, v=self.v, pos=self.pos, layers=layers, kv_heads=heads, group=group,
                      head_dim=64, page_size=page, num_pages=pages)

        def cache(count, per):
            return nexus.Cache(lens=torch.zeros(layers, count, heads, dtype=torch.int32, **dev),
                               seqs=count, capacity=per * page, max_pages_per_seq=per,
                               block_table=torch.full((count, per), -1, dtype=torch.int32, **dev),
                               **common)
        self.prefix, self.cache = cache(2, 8), cache(seqs, per)
        self.pool = nexus.new_pool(self.cache)
        # the prefixes' pages are out of the same pool
        held = nexus.Pool(self.pool.free_pages, self.pool.free_count, _ints([0, 0]))
        self.status = _status()
        self.prompts = [torch.randint(0, V, (n,), generator=g) for n in (61, 37)]
        n = [len(x) for x in self.prompts]
        N = sum(n)
        cu, pos = _ints([0, 0, 0]), torch.empty(N, dtype=torch.int32, **dev)
        nexus.plan(self.prefix, held, _ints(n), cu, self.status, max_tokens=64, token_pos=pos,
                   first_pos=_ints([0, 0]))
        token = torch.cat(self.prompts).to(DEV)
        for l in range(layers):
            q, k, v = self.project(l, token)
            nexus.append(self.prefix, l, None, k, v, pos, None, self.status, max_tokens=64,
                         cu_tokens=cu, rotary=self.rotary)
        self.groups = _ints([0, 3, seqs])

    def project(self, l, token):
        x = self.embed[l].to(DEV)[token.long()]
        HG = self.H * self.G
        return x[:, :HG].contiguous(), x[:, HG:HG + self.H].contiguous(), x[:, HG + self.H:].contiguous()

    def keys64(self, l, token):
        """Keys (not rounded) and values of a sequence's tokens, and the keys' pairs' sizes."""
        x = self.embed[l][token][:, self.H * self.G:].double()
        k = rotate64(x[:, :self.H], range(len(token)), self.freqs, False)
        size = (k[..., :32] ** 2 + k[..., 32:] ** 2).sqrt()
        return k, x[:, self.H:], torch.cat([size, size], -1)


@pytest.mark.parametrize("captured", [False, True])
def test_serving_loop(captured):
    m = Server()
    S, L, H, G, V = m.S, m.L, m.H, m.G, m.V
    rng = np.random.default_rng(7)
    told = [[int(rng.integers(V))] for _ in range(S)]      # tokens of each sequence behind its prompt
    kept = [0] * S                                         # of them, those whose rows the cache holds
    drafts, cap = 3, S * 4
    dev = dict(device=DEV)
    n_new, first = torch.zeros(S, dtype=torch.int32, **dev), torch.zeros(S, dtype=torch.int32, **dev)
    cu = torch.zeros(S + 1, dtype=torch.int32, **dev)
    seq, pos = (torch.zeros(cap, dtype=torch.int32, **dev) for _ in range(2))
    token, out_token = (torch.zeros(cap, dtype=torch.int32, **dev) for _ in range(2))
    p, q = torch.zeros(cap, V, **dev), torch.zeros(cap, V, **dev)
    u, u_draw = torch.zeros(cap, **dev), torch.zeros(S, **dev)
    emitted = torch.zeros(S, dtype=torch.int32, **dev)
    queries = torch.zeros(L, cap, H * G, 64, dtype=BF, **dev)
    seen = torch.zeros_like(queries)
    ws = nexus.alloc_attend_shared_workspace(m.cache, m.prefix, tokens=cap, max_tokens=4,
                                             max_shared=12)
    m.embed_dev = m.embed.to(DEV)

    def step():
        nexus.plan(m.cache, m.pool, n_new, cu, m.status, max_tokens=4, token_seq=seq,
                   token_pos=pos, first_pos=first)
        for l in range(L):
            x = m.embed_dev[l][token.long()]
            nexus.append(m.cache, l, x[:, :H * G], x[:, H * G:H * G + H], x[:, H * G + H:], pos,
                         queries[l], m.status, max_tokens=4, cu_tokens=cu, rotary=m.rotary)
            nexus.attend_shared(m.cache, l, queries[l], seen[l], ws, m.status, prefix=m.prefix,
                                cu_seqs=m.groups, max_tokens=4, max_shared=12, cu_tokens=cu)
        nexus.verify(m.cache, token, p, u, u_draw, out_token, emitted, m.status, max_tokens=4,
                     cu_tokens=cu, q=q)

    graph = None
    for it in range(9):
        n = [int(rng.integers(1, drafts + 2)) for _ in range(S)]
        if it == 5:                                        # sequence 1 ends, and starts over
            n[1] = -1
        bounds = np.concatenate([[0], np.cumsum(np.maximum(n, 0))]).astype(int)
        N = bounds[-1]
        fed, at = [], []
        for s in range(S):
            new = [told[s][-1]] + [int(x) for x in rng.integers(0, V, max(0, n[s] - 1))]
            start = len(m.prompts[0 if s < 3 else 1]) + kept[s]
            fed += new[:max(0, n[s])]
            at += list(range(start, start + max(0, n[s])))
            first[s] = start
        n_new.copy_(_ints(n))
        token.fill_(0)
        token[:N] = _ints(fed)
        pn, _ = _probs(rng, cap, V)
        qn, _ = _probs(rng, cap, V)
        un, dn = rng.random(cap).astype(np.float32) * np.float32(0.2), rng.random(S).astype(np.float32)
        for dst, src in ((p, pn), (q, qn), (u, un), (u_draw, dn)):
            dst.copy_(torch.as_tensor(src))
        if captured and it >= 1:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
            graph.replay()
        else:
            step()
        torch.cuda.synchronize()
        assert int(m.status.item()) == 0
        assert cu.cpu().tolist() == list(bounds)
        assert seq[:N].cpu().tolist() == [s for s in range(S) for _ in range(max(0, n[s]))]
        assert pos[:N].cpu().tolist() == at
        # the rows that the sequence should hold, from its tokens alone; then attention over them
        scale, half = 64 ** -0.5, 2.0 ** -8
        pool = m.k.cpu(), m.v.cpu()
        tables = m.prefix.block_table.cpu().long(), m.cache.block_table.cpu().long()
        for l in range(L):
            for s in range(S):
                if n[s] < 0:                               # (its pages may be others' by now)
                    continue
                a, b, of = bounds[s], bounds[s + 1], 0 if s < 3 else 1
                pr = m.prompts[of]
                text = torch.cat([pr, torch.tensor(told[s][:kept[s]] + fed[a:b], dtype=torch.long)])
                j, own = torch.arange(len(pr)), torch.arange(len(text) - len(pr))
                page = torch.cat([tables[0][of][j // m.page], tables[1][s][own // m.page]])
                slot = torch.cat([j, own]) % m.page
                k, v = (x[l, page, :, slot].double() for x in pool)
                want_k, want_v, size = m.keys64(l, text)
                # one rounding of a rotated pair, and some 16 fp32 ones before it
                assert torch.all((k - want_k).abs() <= half * want_k.abs() + 2.0 ** -20 * size)
                assert torch.equal(v, want_v)
                for i in range(b - a):
                    T = len(text) - (b - a) + i + 1
                    for h in range(H):
                        qi = queries[l, a + i, h * G:(h + 1) * G].cpu()
                        ro, _, A, big = attend64(qi, k[:T, h], v[:T, h], [T] * G, scale)
                        got = seen[l, a + i, h * G:(h + 1) * G].cpu().double()
                        dx = scale * big * 2.0 ** -24 * 72
                        tol = half * ro.abs() + (half + 2.0 ** -20 + 2 * dx)[:, None] * A
                        assert torch.all((got - ro).abs() <= tol), (it, l, s, i, h)
        want = B.verify_plain(fed, pn, qn, un, dn, list(bounds))
        assert out_token[:N].cpu().tolist() == want[0] and emitted.cpu().tolist() == want[1]
        for s in range(S):
            if n[s] < 0:
                told[s], kept[s] = [3], 0
                continue
            a, e = bounds[s], want[1][s]
            told[s] = told[s][:kept[s]] + [fed[a]] + want[0][a:a + e]
            kept[s] += e
        lens = m.cache.lens.cpu()
        assert torch.equal(lens, torch.tensor(kept, dtype=torch.int32)[None, :, None].expand(L, S, H))
    # nobody holds a page twice
    held = m.pool.held.cpu().tolist()
    mine = [x for s in range(S) for x in m.cache.block_table[s, :held[s]].cpu().tolist()]
    pre = m.prefix.block_table[:, :].cpu()
    pre = pre[0, :-(-61 // 8)].tolist() + pre[1, :-(-37 // 8)].tolist()
    free = m.pool.free_pages[:int(m.pool.free_count.item())].cpu().tolist()
    assert sorted(mine + pre + free) == list(range(m.cache.num_pages))


def test_calls_on_another_stream():
    own, pre = _pair("bf16", 6, 1, 40, 700)
    cache, prefix, st = own.device_cache(), pre.device_cache(), _status()
    q = torch.randn(6, 8, 128, generator=own.g).to(DEV, BF)
    ws = nexus.alloc_attend_shared_workspace(cache, prefix, tokens=6, max_tokens=1, max_shared=6)
    a, b = torch.empty_like(q), torch.empty_like(q)
    nexus.attend_shared(cache, 0, q, a, ws, st, prefix=prefix, max_tokens=1, max_shared=6)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    nexus.attend_shared(cache, 0, q, b, ws, st, prefix=prefix, max_tokens=1, max_shared=6,
                        stream=other)
    other.synchronize()
    assert torch.equal(a, b) and int(st.item()) == 0
    bare = _bare_cache(1, 2, 1, 50, lens=_ints([[[5], [6]]]))
    cu, pos = _ints([0, 0, 0]), _ints([0, 0])
    out, em = _ints([0, 0]), _ints([0, 0])
    n, first = _ints([1, 1]), _ints([4, 5])
    p = torch.full((2, 8), 0.125, device=DEV)
    u = torch.zeros(2, device=DEV)
    with torch.cuda.stream(other):
        other.wait_stream(torch.cuda.default_stream())
        nexus.plan(bare, None, n, cu, st, max_tokens=1, token_pos=pos, first_pos=first)
        nexus.verify(bare, out.clone(), p, u, u, out, em, st, max_tokens=1, cu_tokens=cu)
    other.synchronize()
    assert int(st.item()) == 0 and pos.cpu().tolist() == [4, 5] and em.cpu().tolist() == [1, 1]


@pytest.mark.parametrize("prefix_rows,seqs", [(40, 6), (4200, 24), (300, 40)])
def test_steps_of_many_layers_without_a_pause(prefix_rows, seqs):
    # append and attend_shared of three layers and five steps in a row, one workspace, against the
    # same with a pause behind every call; then from a graph. Nothing may run ahead of what it reads
    # or overwrite what somebody still reads: the bits are the same.
    def run(how):
        own, pre = _pair("bf16", seqs, 1, 30, prefix_rows, layers=3, page=16)
        g = torch.Generator(device=DEV).manual_seed(3)
        own = Case(seqs=seqs, kv_heads=2, group=4, layers=3, page=16, capacity=64, lens=30, seed=1)
        cache, prefix, st = own.device_cache(), pre.device_cache(), _status()
        cache.k.nan_to_num_(), cache.v.nan_to_num_()
        x = torch.randn(5, 3, seqs, 12, 128, generator=g, device=DEV).to(BF)
        pos = torch.full((seqs,), 7, dtype=torch.int32, device=DEV)
        rot = torch.empty(seqs, 8, 128, dtype=BF, device=DEV)
        out = torch.zeros(5, 3, seqs, 8, 128, dtype=BF, device=DEV)
        ws = nexus.alloc_attend_shared_workspace(cache, prefix, tokens=seqs, max_tokens=1,
                                                 max_shared=seqs)

        def steps():
            for i in range(5):
                for l in range(3):
                    p = x[i, l]
                    nexus.append(cache, l, p[:, :8], p[:, 8:10], p[:, 10:], pos, rot, st, max_tokens=1)
                    if how == "paused":
                        torch.cuda.synchronize()
                    nexus.attend_shared(cache, l, rot, out[i, l], ws, st, prefix=prefix, max_tokens=1,
                                        max_shared=seqs)
                    if how == "paused":
                        torch.cuda.synchronize()
        if how == "graph":
            lens = cache.lens.clone()
            graph = torch.cuda.CUDAGraph()
            steps()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                steps()
            for _ in range(3):
                cache.lens.copy_(lens)
                out.zero_()
                graph.replay()
        else:
            steps()
        torch.cuda.synchronize()
        assert int(st.item()) == 0 and torch.all(cache.lens == 35)
        return out
    want = run("paused")
    assert torch.all(torch.isfinite(want)) and want.abs().max() > 0
    for how in ("straight", "straight", "graph"):
        assert torch.equal(run(how), want), how
