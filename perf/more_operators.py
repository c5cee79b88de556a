"""What is measured of the operators around a batch of sequences that decode from a shared pool.

A serving step over the library's KV cache has three ends besides ``append`` and ``attend``:
``plan`` deals out the pool's pages to the sequences for the tokens that they bring next and
lays out the batch, ``attend_shared`` attends over a prefix that many sequences share (read
once for all of them) and over each sequence's own rows, and ``verify`` judges drafted tokens
against the model's probabilities, draws the token behind the last one kept and takes the
rejected ones back from the cache.

``run`` is one pass through one of the three, by elementary torch operations where ``own`` is
false and by the library's entry points where it is true.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 32
UNIT = 42                    # weights of a draw are counted in units of 2^-42

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

#: What a case holds unless it says otherwise.
PLAN = {"op": "plan", "layers": 32, "seqs": 16, "kv_heads": 8, "page": 16, "rows": 1024, "tokens": 1,
        "churn": 0.0}
VERIFY = {"op": "verify", "layers": 32, "seqs": 1, "kv_heads": 8, "vocab": 32000, "dtype": "f32",
          "tokens": 5, "ragged": False, "drafted": True, "image": False}
SHARED = {"op": "shared", "prefixes": 1, "seqs": 16, "loose": 0, "kv_heads": 8, "group": 4, "d": 128,
          "dtype": "bf16", "page": 0, "prefix_rows": 4096, "rows": 128, "ragged": False,
          "tokens": 1, "causal": True, "image": "none"}


def listed():
    return [
        # one more token of each of 16 sequences: now and then one of them needs a page
        {"name": "plan_decode", **PLAN},
        # 256 sequences of all lengths, a third of which end, arrive or were just evicted
        {"name": "plan_churn", **PLAN, "seqs": 256, "rows": 8192, "tokens": 6, "churn": 0.35},
        # prompts of up to 2048 tokens arrive in 96 places at once
        {"name": "plan_prompts", **PLAN, "seqs": 96, "page": 32, "rows": 2048, "tokens": 2048,
         "churn": 0.6},
        # four drafted tokens of one sequence
        {"name": "verify_one", **VERIFY},
        # five drafted tokens of 64 sequences, a large vocabulary, the image follows
        {"name": "verify_batch", **VERIFY, "seqs": 64, "vocab": 131072, "tokens": 6, "image": True},
        # drafts without probabilities of their own (looked up, not drawn), bf16, odd rows
        {"name": "verify_looked_up", **VERIFY, "seqs": 200, "vocab": 50257, "dtype": "bf16",
         "tokens": 8, "ragged": True, "drafted": False},
        # no drafts at all: one token drawn for each of 256 sequences
        {"name": "verify_draw", **VERIFY, "seqs": 256, "vocab": 65536, "tokens": 1,
         "drafted": False},
        # a few sequences of a small fp32 head behind a short prefix
        {"name": "shared_small_f32", **SHARED, "seqs": 4, "kv_heads": 1, "group": 1, "d": 64,
         "dtype": "f32", "prefix_rows": 500, "rows": 37},
        # one decoded token of 16 sequences behind the same instructions
        {"name": "shared_instructions", **SHARED},
        # one decoded token of 64 sequences over one long document, own rows ragged, paged
        {"name": "shared_document", **SHARED, "seqs": 64, "prefix_rows": 32768, "rows": 1024,
         "page": 16, "ragged": True},
        # a few drafted tokens each of 48 sequences over 3 prompts, some sequences without one
        {"name": "shared_drafts", **SHARED, "prefixes": 3, "seqs": 48, "loose": 5,
         "prefix_rows": 8704, "rows": 600, "tokens": 5, "page": 32, "ragged": True},
        # the document again, its rows from the 8-bit image
        {"name": "shared_document8", **SHARED, "seqs": 64, "prefix_rows": 32768, "rows": 1024,
         "page": 32, "ragged": True, "image": "prefix"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "verify", "verify", "shared", "shared", "shared"])
    if op == "plan":
        c = dict(PLAN)
        c["layers"] = _log(rng, 1, 64)
        c["seqs"] = _log(rng, 1, 1024)
        c["kv_heads"] = rng.choice([1, 2, 5, 8])
        c["page"] = rng.choice([8, 16, 32, 64, 128])
        c["rows"] = _log(rng, 1, 16384)
        c["tokens"] = rng.choice([1, _log(rng, 2, 16), _log(rng, 2, max(2, 65536 // c["seqs"]))])
        c["churn"] = rng.choice([0.0, 0.1, 0.5])
    elif op == "verify":
        c = dict(VERIFY)
        c["layers"] = _log(rng, 1, 64)
        c["seqs"] = _log(rng, 1, 512)
        c["kv_heads"] = rng.choice([1, 2, 5, 8])
        c["tokens"] = rng.randint(1, 9)
        most = 64 * 6 * 131072 // (c["seqs"] * c["tokens"])
        c["vocab"] = _log(rng, min(most, 250), min(most, 200000))
        c["dtype"] = rng.choice(["f32", "f32", "bf16"])
        c["ragged"] = rng.random() < 0.5
        c["drafted"] = rng.random() < 0.7
        c["image"] = rng.random() < 0.4
    else:
        c = dict(SHARED)
        c["seqs"] = _log(rng, 1, 128)
        c["prefixes"] = rng.choice([1, 1, min(c["seqs"], rng.randint(2, 8))])
        c["loose"] = rng.choice([0, 0, c["seqs"] // 5])
        c["kv_heads"] = rng.choice([1, 2, 5, 8])
        c["group"] = rng.choice([1, 2, 3, 4, 6, 8])
        c["d"] = rng.choice([64, 128, 128])
        c["dtype"] = rng.choice(["bf16", "bf16", "bf16", "f32"])
        c["page"] = rng.choice([0, 0, 8, 16, 32, 64, 128])
        c["ragged"] = rng.random() < 0.6
        c["tokens"] = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 2, 128)])
        c["causal"] = rng.random() < 0.8
        if c["dtype"] == "bf16":
            c["image"] = rng.choice(["none", "none", "prefix", "both"])
        c["tokens"] = min(c["tokens"], max(1, 4096 // c["seqs"]))
        heads = c["kv_heads"] * c["group"] * c["tokens"] * c["seqs"]
        flops = 64 * 32 * 32768 // heads // (4 if c["dtype"] == "f32" else 1)
        held = 2 * 8 * 32768 // (c["prefixes"] * c["kv_heads"])
        c["prefix_rows"] = _log(rng, 1, max(1, min(65536, flops, held)))
        c["rows"] = _log(rng, 1, max(1, min(4096, flops, 65536 // c["seqs"])))
    return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 29)
    h = np.random.default_rng([int(seed), case["seqs"], case["tokens"], case["kv_heads"]])
    st = {"case": case}
    {"plan": _prepare_plan, "verify": _prepare_verify, "shared": _prepare_shared}[case["op"]](
        st, case, dev, g, h)
    return st


def _ints(x, dev):
    return torch.as_tensor(np.ascontiguousarray(x).astype(np.int32), device=dev)


def _counts(c):
    """Tokens of each sequence, by the case alone: the outputs' shapes go by them."""
    S, M = c["seqs"], c["tokens"]
    if not c["ragged"] or M == 1:
        return np.full(S, M)
    n = np.random.default_rng([S, M]).integers(0, M + 1, S)
    n[0] = M
    return n


def _cu(n):
    return np.concatenate([[0], np.cumsum(n)])


def _prepare_plan(st, c, dev, g, h):
    S, L, H, page = c["seqs"], c["layers"], c["kv_heads"], c["page"]
    per = -(-(c["rows"] + 2 * c["tokens"]) // page)      # pages of a sequence, at most
    rows = h.integers(c["rows"] // 16, c["rows"] + 1, S)
    kind = h.random(S)
    churn = kind < c["churn"]
    came = churn & (kind < c["churn"] * 0.4)             # a prompt in an empty place
    ended = churn & ~came & (kind < c["churn"] * 0.7)
    evicted = churn & ~came & ~ended                     # holds pages for more than it has
    rows[came] = 0
    held = -(-rows // page)
    rows[evicted] = rows[evicted] // 5
    n = h.integers(1, c["tokens"] + 1, S)
    if c["churn"]:                                       # those that go on bring a few tokens
        n[~came] = np.minimum(n[~came], 8)
    n[ended] = -1
    lens = h.integers(0, 1 << 30, (L, S, H)) % (rows[None, :, None] // 2 + 1) \
        + (rows - rows // 2)[None, :, None]
    lens[h.integers(0, L, S), np.arange(S), h.integers(0, H, S)] = rows
    pages = S * per + 5
    order = h.permutation(pages)
    table = h.integers(0, pages, (S, per))               # what lies behind held means nothing
    at = 0
    for s in range(S):
        table[s, :held[s]] = order[at:at + held[s]]
        at += held[s]
    free = np.zeros(pages, np.int64)
    free[:pages - at] = order[at:]
    tokens = S * c["tokens"]
    st.update(pages=pages, per=per, tokens=tokens, table=_ints(table, dev), free=_ints(free, dev),
              free_in=_ints([pages - at], dev), free_count=_ints([0], dev), held_in=_ints(held, dev),
              held=_ints(held, dev), n=_ints(n, dev), lens=_ints(lens, dev),
              first_pos=_ints(h.integers(0, 1 << 20, S), dev),
              cu=torch.zeros(S + 1, dtype=torch.int32, device=dev),
              token_seq=torch.full((tokens,), -1, dtype=torch.int32, device=dev),
              token_pos=torch.full((tokens,), -1, dtype=torch.int32, device=dev))


def _prepare_verify(st, c, dev, g, h):
    S, L, H, V = c["seqs"], c["layers"], c["kv_heads"], c["vocab"]
    n = _counts(c)
    N = int(n.sum())

    def normal(*shape):
        return torch.empty(shape, device=dev).normal_(generator=g)

    # a model's distributions: a few likely tokens and a long tail; the draft's are near them
    logits = normal(N, V) * 2.5
    p = torch.softmax(logits, -1)
    if c["drafted"]:
        q = torch.softmax(logits.add_(normal(N, V), alpha=0.6), -1)
    del logits
    p = p.to(DTYPES[c["dtype"]])
    q = q.to(DTYPES[c["dtype"]]) if c["drafted"] else None
    # row i's draft is token i + 1 of its sequence; the first token of each is the last one known
    drafts = torch.multinomial((p if q is None else q).float(), 1, generator=g)[:, 0].int()
    token = torch.cat([drafts[:1], drafts[:-1]])
    st.update(n=N, p=p, q=q, token=token, max_tokens=c["tokens"],
              cu=None if (n == c["tokens"]).all() else _ints(_cu(n), dev), bounds=_cu(n),
              u=torch.rand(N, generator=g, device=dev),
              u_draw=torch.rand(S, generator=g, device=dev),
              out=torch.zeros(N, dtype=torch.int32, device=dev),
              emitted=torch.zeros(S, dtype=torch.int32, device=dev))
    lens = _ints(h.integers(64, 4096, (L, S, H)), dev)
    st.update(lens_in=lens, lens=lens.clone(), rows8=lens // BLOCK * BLOCK)


def _prepare_shared(st, c, dev, g, h):
    S, P, H, G, d, M = (c["seqs"], c["prefixes"], c["kv_heads"], c["group"], c["d"], c["tokens"])
    dt, page = DTYPES[c["dtype"]], c["page"]

    def normal(*shape, dtype=dt):
        return torch.empty(shape, device=dev, dtype=dtype).normal_(generator=g)

    n = _counts(c)
    N = int(n.sum())
    cuts = np.random.default_rng([S, P, 3]).integers(0, S - c["loose"] + 1, P - 1)
    groups = np.concatenate([[0], np.sort(cuts), [S - c["loose"]]])
    st.update(n=N, cu=None if (n == M).all() else _ints(_cu(n), dev), bounds=_cu(n), groups=groups,
              cu_seqs=_ints(groups, dev),
              max_shared=max(1, int(max(_cu(n)[groups[1:]] - _cu(n)[groups[:-1]]))))

    def lengths(count, most, least):
        if not c["ragged"]:
            return np.full((1, count, H), max(most, least))
        x = h.integers(most // 2, most + 1, (1, count, H))
        x.reshape(-1)[0] = most
        return np.maximum(x, least)

    # own rows: what was decoded behind the prefix, the new tokens among them
    lens = {"prefix": lengths(P, c["prefix_rows"], 0), "own": lengths(S, c["rows"], M)}
    block = min(BLOCK, page) if page else BLOCK
    if page:
        per = {k: -(-int(x.max()) // page) for k, x in lens.items()}
        pages = P * per["prefix"] + S * per["own"] + 3
        order = h.permutation(pages)
        st["table_prefix"] = _ints(order[:P * per["prefix"]].reshape(P, -1), dev)
        st["table_own"] = _ints(order[P * per["prefix"]:-3].reshape(S, -1), dev)
        shapes = {"pool": (1, pages, H, page)}
        st["pages"] = pages
    else:
        cap = {k: -(-int(x.max()) // BLOCK) * BLOCK for k, x in lens.items()}
        shapes = {"prefix": (1, P, H, cap["prefix"]), "own": (1, S, H, cap["own"])}
    for part, shape in shapes.items():
        for name in ("k", "v"):
            x = normal(*shape, d)
            if c["image"] != "none":                     # heads and rows differ in size
                x *= torch.exp(0.5 * normal(*shape, 1, dtype=torch.float32)).to(dt)
                most = x.float().unflatten(3, (-1, block)).abs().amax((4, 5))
                m, e = torch.frexp(most)
                e = torch.where(m > 0.875, e - 8, e - 9)
                scale = torch.ldexp(torch.ones_like(most), e)
                st[f"{name}_scale_{part}"] = scale
                st[f"{name}8_{part}"] = (x.float() / scale.repeat_interleave(block, 3)[..., None]) \
                    .clamp(-448, 448).to(torch.float8_e4m3fn)
            st[f"{name}_{part}"] = x
        st[f"pos_{part}"] = torch.zeros(shape, dtype=torch.int32, device=dev)
    for part in ("prefix", "own"):
        st[f"lens_{part}"] = _ints(lens[part], dev)
        here = c["image"] == "both" or c["image"] == part
        st[f"rows8_{part}"] = st[f"lens_{part}"] // block * block if here else None
        if page:
            for name in ("k", "v", "k8", "v8", "k_scale", "v_scale", "pos"):
                if f"{name}_pool" in st:
                    st[f"{name}_{part}"] = st[f"{name}_pool"]
    # queries that look for one of the prefix's rows each, next to everything else
    st["q"] = normal(N, H * G, d)
    if groups[-1] > 0 and N:
        seq = np.repeat(np.arange(S), n)
        group = np.searchsorted(groups, seq, side="right") - 1
        group = torch.as_tensor(np.minimum(group, P - 1), device=dev)
        ln = st["lens_prefix"][0][group].clamp(min=1).float()
        aim = (torch.rand(N, H, generator=g, device=dev) * ln).long()
        head = torch.arange(H, device=dev).expand(N, H)
        where = group[:, None].expand(N, H)
        if page:
            hub = st["k_pool"][0][st["table_prefix"].long()[where, aim // page], head, aim % page]
        else:
            hub = st["k_prefix"][0][where, head, aim]
        hub = hub.float()
        hub = 6 * hub / hub.norm(dim=-1, keepdim=True)
        st["q"] += hub.repeat_interleave(G, dim=1).to(dt)
    st["out"] = torch.zeros(N, H * G, d, device=dev, dtype=dt)
    st["lse"] = torch.zeros(N, H * G, device=dev)


# ---------------------------------------------------------------------------
# The operators
# ---------------------------------------------------------------------------

def _handle(st):
    """The objects that a user's program makes once for its buffers."""
    if "handle" in st:
        return st["handle"]
    from streaming_kv_cache_step_gb300 import nexus
    c = st["case"]
    dev = torch.device("cuda")
    # for the keys and values of a cache, which plan and verify do not touch
    some = torch.zeros(64, dtype=torch.bfloat16, device=dev)
    if c["op"] == "plan":
        cache = nexus.Cache(k=some, v=some, pos=some.int(), lens=st["lens"], layers=c["layers"],
                            seqs=c["seqs"], kv_heads=c["kv_heads"], group=4, head_dim=128,
                            capacity=st["per"] * c["page"], page_size=c["page"],
                            num_pages=st["pages"], max_pages_per_seq=st["per"],
                            block_table=st["table"])
        more = nexus.Pool(free_pages=st["free"], free_count=st["free_count"], held=st["held"])
    elif c["op"] == "verify":
        cache = nexus.Cache(k=some, v=some, pos=some.int(), lens=st["lens"], layers=c["layers"],
                            seqs=c["seqs"], kv_heads=c["kv_heads"], group=4, head_dim=128,
                            capacity=4096)
        more = None
        if c["image"]:
            scales = torch.ones(cache.n_slices * 4096 // BLOCK, device=dev)
            more = nexus.Image(k=some.to(torch.float8_e4m3fn), v=some.to(torch.float8_e4m3fn),
                               k_scale=scales, v_scale=scales, rows=st["rows8"])
    else:
        made = []
        for part, count in (("own", c["seqs"]), ("prefix", c["prefixes"])):
            page = c["page"]
            per = st[f"table_{part}"].shape[1] if page else 0
            cap = per * page if page else st[f"k_{part}"].shape[3]
            made.append(nexus.Cache(
                k=st[f"k_{part}"], v=st[f"v_{part}"], pos=st[f"pos_{part}"],
                lens=st[f"lens_{part}"], layers=1, seqs=count, kv_heads=c["kv_heads"],
                group=c["group"], head_dim=c["d"], capacity=cap, page_size=page,
                num_pages=st["pages"] if page else 0, max_pages_per_seq=per,
                block_table=st[f"table_{part}"] if page else None))
            im = None
            if st[f"rows8_{part}"] is not None:
                im = nexus.Image(k=st[f"k8_{part}"], v=st[f"v8_{part}"],
                                 k_scale=st[f"k_scale_{part}"], v_scale=st[f"v_scale_{part}"],
                                 rows=st[f"rows8_{part}"])
            made.append(im)
        cache, image, prefix, prefix_image = made
        ws = nexus.alloc_attend_shared_workspace(cache, prefix, tokens=st["n"],
                                                 max_tokens=c["tokens"],
                                                 max_shared=st["max_shared"])
        more = image, prefix, prefix_image, ws
    st["handle"] = nexus, cache, more, nexus.new_status(dev)
    return st["handle"]


def run(state):
    st, c = state, state["case"]
    if own:
        nexus, cache, more, status = _handle(st)
        if c["op"] == "plan":
            nexus.plan(cache, more, st["n"], st["cu"], status, max_tokens=c["tokens"],
                       token_seq=st["token_seq"], token_pos=st["token_pos"],
                       first_pos=st["first_pos"], held_in=st["held_in"],
                       free_count_in=st["free_in"])
        elif c["op"] == "verify":
            nexus.verify(cache, st["token"], st["p"], st["u"], st["u_draw"], st["out"],
                         st["emitted"], status, max_tokens=c["tokens"], cu_tokens=st["cu"],
                         q=st["q"], lens_in=st["lens_in"], image=more)
        else:
            image, prefix, prefix_image, ws = more
            nexus.attend_shared(cache, 0, st["q"], st["out"], ws, status, prefix=prefix,
                                cu_seqs=st["cu_seqs"], max_shared=st["max_shared"],
                                max_tokens=c["tokens"], cu_tokens=st["cu"], causal=c["causal"],
                                lse=st["lse"], image=image, prefix_image=prefix_image)
    else:
        {"plan": _plan_plain, "verify": _verify_plain, "shared": _shared_plain}[c["op"]](st)
    if c["op"] == "plan":
        return {k: st[k] for k in ("table", "free", "free_count", "held", "lens", "cu",
                                   "token_seq", "token_pos")}
    if c["op"] == "verify":
        return {k: st[k] for k in ("out", "emitted", "lens", "rows8")}
    return {"out": st["out"], "lse": st["lse"]}


def _plan_plain(st):
    c, n = st["case"], st["n"].long()
    S, per, dev = c["seqs"], st["per"], st["n"].device
    ended = n < 0
    n = n.clamp(min=0)
    rows = st["lens"].amax((0, 2)).long().masked_fill(ended, 0)
    need = (rows + n + c["page"] - 1) // c["page"]
    held = st["held_in"].long()
    gives, takes = (held - need).clamp(min=0), (need - held).clamp(min=0)
    first_free = st["free_in"].long()
    entry = torch.arange(per, device=dev).expand(S, per)
    # pages given back go on top of the free ones, in the order of sequences
    out = (entry >= need[:, None]) & (entry < held[:, None])
    s, e = out.nonzero(as_tuple=True)
    at = first_free + (gives.cumsum(0) - gives)[s] + e - need[s]
    st["free"][at] = st["table"][s, e]
    top = first_free + gives.sum()
    # and pages are taken from there, the last one first
    new = (entry >= held[:, None]) & (entry < need[:, None])
    s, e = new.nonzero(as_tuple=True)
    at = top - 1 - (takes.cumsum(0) - takes)[s] - (e - held[s])
    st["table"][s, e] = st["free"][at]
    st["free_count"].copy_(top - takes.sum())
    st["held"].copy_(need)
    st["lens"].copy_(torch.where(ended[None, :, None], 0, st["lens"]))
    ends = n.cumsum(0)
    st["cu"][0] = 0
    st["cu"][1:] = ends
    i = torch.arange(int(ends[-1]), device=dev)
    s = torch.searchsorted(ends, i, right=True)
    st["token_seq"][:i.numel()] = s.int()
    st["token_pos"][:i.numel()] = (st["first_pos"].long()[s] + i - (ends - n)[s]).int()


def _verify_plain(st):
    c, dev = st["case"], st["p"].device
    S, V, N = c["seqs"], c["vocab"], st["n"]
    cu = torch.as_tensor(st["bounds"], device=dev) if st["cu"] is None else st["cu"].long()
    a, b = cu[:-1], cu[1:]
    row = torch.arange(N, device=dev)
    seq = torch.searchsorted(cu, row, right=True) - 1
    nxt = (row + 1).clamp(max=N - 1)
    x = st["token"].long()[nxt][:, None]
    px = st["p"].gather(1, x)[:, 0].double()
    qx = torch.ones_like(px) if st["q"] is None else st["q"].gather(1, x)[:, 0].double()
    drafted = row + 1 < b[seq]
    bad = drafted & ~(st["u"].double() * qx < px)
    # the first row whose draft goes: the last row if none does
    stop = torch.where(bad | ~drafted, row, N)
    r = torch.full((S,), N, device=dev).scatter_reduce(0, seq, stop, "amin")
    some = b > a
    at = r.clamp(max=N - 1)
    w = st["p"][at].float()
    rest = (r + 1 < b)[:, None]
    if st["q"] is None:
        gone = torch.zeros_like(w).scatter_(1, st["token"].long()[nxt[at]][:, None], 1.0)
        gone = (gone > 0) & rest
        w = torch.where(gone, 0.0, w)
    else:
        w = torch.where(rest, (w - st["q"][at].float()).clamp(min=0), w)
    sums = (w.double() * 2.0 ** UNIT).long().cumsum(1)
    total = sums[:, -1]
    u = (st["u_draw"].double() * 2.0 ** 31).long()
    t = u * (total >> 31) + (u * (total & 0x7FFFFFFF) >> 31)
    drawn = torch.searchsorted(sums, t[:, None], right=True)[:, 0]
    kept = torch.where(row < r[seq], st["token"].long()[nxt], -1)
    kept[at[some]] = drawn[some]
    st["out"].copy_(kept)
    st["emitted"].copy_(torch.where(some, r - a + 1, 0))
    lens = st["lens_in"] - torch.where(some, b - 1 - r, 0)[None, :, None].int()
    st["lens"].copy_(lens)
    if c["image"]:
        st["rows8"].copy_(torch.minimum(st["rows8"], lens // BLOCK * BLOCK))


def _rows(st, part):
    """Keys and values of a cache, [count, kv_heads, capacity, d] in 32 bits, those that the
    image holds from there."""
    c = st["case"]
    page = c["page"]
    table = st[f"table_{part}"].long() if page else None

    def whole(name):
        x = st[f"{name}_{part}"][0]
        if page:
            x = x[table].transpose(1, 2)
            x = x.reshape(*x.shape[:2], -1, *x.shape[4:])
        return x

    got = []
    for name in ("k", "v"):
        x = whole(name).float()
        if st[f"rows8_{part}"] is not None:
            b = min(BLOCK, page) if page else BLOCK
            y = whole(name + "8").float() * whole(name + "_scale").repeat_interleave(b, 2)[..., None]
            held = torch.arange(x.shape[2], device=x.device) < st[f"rows8_{part}"][0][..., None]
            x = torch.where(held[..., None], y, x)
        got.append(x)
    return got


def _shared_plain(st):
    c = st["case"]
    S, H, G, d, M, N = c["seqs"], c["kv_heads"], c["group"], c["d"], c["tokens"], st["n"]
    dev, scale = st["q"].device, 1 / math.sqrt(c["d"])
    q = st["q"].float().reshape(N, H, G, d)
    inf = math.inf

    def partial(x, v):
        top = x.amax(-1, keepdim=True)
        e = torch.exp(x - torch.where(top > -inf, top, 0.0))
        return top[..., 0], e.sum(-1), torch.matmul(e, v)

    # the prefixes: the tokens of all their sequences at once
    m1 = torch.full((N, H, G), -inf, device=dev)
    z1, o1 = torch.zeros(N, H, G, device=dev), torch.zeros(N, H, G, d, device=dev)
    k, v = _rows(st, "prefix")
    for p in range(c["prefixes"]):
        a, b = st["bounds"][st["groups"][p]], st["bounds"][st["groups"][p + 1]]
        if a == b:
            continue
        x = q[a:b].transpose(0, 1).reshape(H, -1, d)
        x = torch.matmul(x, k[p].transpose(-1, -2)) * scale
        off = torch.arange(k.shape[2], device=dev) >= st["lens_prefix"][0, p][:, None]
        x.masked_fill_(off[:, None], -inf)
        m, z, o = partial(x, v[p].masked_fill(off[..., None], 0))
        m1[a:b] = m.reshape(H, -1, G).transpose(0, 1)
        z1[a:b] = z.reshape(H, -1, G).transpose(0, 1)
        o1[a:b] = o.reshape(H, -1, G, d).transpose(0, 1)
    # their own rows
    k, v = _rows(st, "own")
    cu = torch.as_tensor(st["bounds"], device=dev)
    n = cu[1:] - cu[:-1]
    i = torch.arange(M, device=dev)
    here = i < n[:, None]
    tok = (cu[:-1, None] + i).clamp(max=max(0, N - 1))
    x = q[tok].permute(0, 2, 1, 3, 4).reshape(S, H, M * G, d)
    x = torch.matmul(x, k.transpose(-1, -2)) * scale
    lens = st["lens_own"][0].long()
    last = (n[:, None] - 1 - i) if c["causal"] else torch.zeros_like(here, dtype=torch.long)
    limit = (lens[:, :, None] - last[:, None]).clamp(min=0).repeat_interleave(G, dim=2)
    slot = torch.arange(k.shape[2], device=dev)
    x.masked_fill_(slot >= limit[..., None], -inf)
    m2, z2, o2 = partial(x, v.masked_fill((slot >= lens[..., None])[..., None], 0))
    m2, z2 = (y.reshape(S, H, M, G).transpose(1, 2)[here] for y in (m2, z2))
    o2 = o2.reshape(S, H, M, G, d).transpose(1, 2)[here]
    top = torch.maximum(m1, m2)
    ref = torch.where(top > -inf, top, 0.0)
    f1, f2 = torch.exp(m1 - ref), torch.exp(m2 - ref)
    z = z1 * f1 + z2 * f2
    o = (o1 * f1[..., None] + o2 * f2[..., None]) / torch.where(z > 0, z, 1.0)[..., None]
    st["out"].copy_(o.reshape(N, H * G, d))
    st["lse"].copy_((top + torch.log(z)).reshape(N, H * G))


# ---------------------------------------------------------------------------
# What a pass cannot do without, and the definition in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    c = case
    S = c["seqs"]
    if c["op"] == "plan":
        most = min(c["tokens"], 8) if c["churn"] else c["tokens"]
        tokens = S * (c["churn"] * 0.4 * (c["tokens"] + 1) / 2 + (1 - c["churn"] * 0.7) * (most + 1) / 2)
        moved = S * c["churn"] * (0.12 * c["tokens"] + 0.6 * c["rows"] / 2) / c["page"] + \
            tokens / c["page"]
        return {"bytes": 4 * (c["layers"] * S * c["kv_heads"] + 6 * S + 2 * tokens + 2 * moved),
                "flops": c["layers"] * S * c["kv_heads"] + 4 * tokens}
    n = _counts(c)
    if c["op"] == "verify":
        size = 4 if c["dtype"] == "f32" else 2
        some = int((n > 0).sum())
        cache = c["layers"] * S * c["kv_heads"]
        # one row of p, and of q where there are drafts, for each sequence
        rows = some * (2 if c["drafted"] and c["tokens"] > 1 else 1)
        return {"bytes": rows * c["vocab"] * size + int(n.sum()) * (12 + 2 * size) + 8 * cache,
                "flops": some * c["vocab"] * 3}
    H, G, d = c["kv_heads"], c["group"], c["d"]
    size = 4 if c["dtype"] == "f32" else 2
    mean = 0.75 if c["ragged"] else 1.0
    code = 1 + 4 / BLOCK / d
    size_p = code if c["image"] in ("prefix", "both") else size
    size_o = code if c["image"] == "both" else size
    prefix, rows = mean * c["prefix_rows"], max(mean * c["rows"], c["tokens"])
    tokens = int(n.sum())
    shared = int(_cu(n)[S - c["loose"]])
    return {"bytes": 2 * H * d * (c["prefixes"] * prefix * size_p + S * rows * size_o) +
            tokens * H * G * (2 * d * size + 4),
            "flops": 4 * d * H * G * (shared * prefix + tokens * rows)}


def exact(case, seed):
    st = prepare(case, seed)
    return {"plan": _plan_exact, "verify": _verify_exact, "shared": _shared_exact}[case["op"]](st)


def _plan_exact(st):
    """Sequence by sequence, page by page."""
    c = st["case"]
    lens, held, n = (st[k].cpu().numpy().copy() for k in ("lens", "held_in", "n"))
    table, free = st["table"].cpu().numpy().copy(), st["free"].cpu().numpy().copy()
    first = st["first_pos"].cpu().numpy()
    token_seq, token_pos = st["token_seq"].cpu().numpy(), st["token_pos"].cpu().numpy()
    top = int(st["free_in"])
    wants = []
    for s in range(c["seqs"]):
        if n[s] < 0:
            lens[:, s] = 0
        wants.append(-(-(int(lens[:, s].max()) + max(0, int(n[s]))) // c["page"]))
    for s, want in enumerate(wants):
        for e in range(want, held[s]):
            free[top] = table[s, e]
            top += 1
    cu = [0]
    for s, want in enumerate(wants):
        for e in range(held[s], want):
            top -= 1
            table[s, e] = free[top]
        for i in range(max(0, int(n[s]))):
            token_seq[cu[-1] + i], token_pos[cu[-1] + i] = s, first[s] + i
        cu.append(cu[-1] + max(0, int(n[s])))
    dev = st["n"].device
    return {"table": _ints(table, dev), "free": _ints(free, dev), "free_count": _ints([top], dev),
            "held": _ints(wants, dev), "lens": _ints(lens, dev), "cu": _ints(cu, dev),
            "token_seq": _ints(token_seq, dev), "token_pos": _ints(token_pos, dev)}


def _verify_exact(st):
    """Sequence by sequence, draft by draft."""
    c, dev = st["case"], st["p"].device
    token, u = st["token"].cpu().numpy(), st["u"].cpu().numpy().astype(np.float64)
    u_draw = st["u_draw"].cpu().numpy().astype(np.float64)
    out, emitted = np.full(st["n"], -1), np.zeros(c["seqs"], np.int64)
    lens = st["lens_in"].cpu().numpy().copy()
    for s in range(c["seqs"]):
        a, b = int(st["bounds"][s]), int(st["bounds"][s + 1])
        if a == b:
            continue
        i = a
        while i + 1 < b:
            x = int(token[i + 1])
            q = 1.0 if st["q"] is None else float(st["q"][i, x])
            if not u[i] * q < float(st["p"][i, x]):
                break
            out[i] = x
            i += 1
        w = st["p"][i].float().cpu().numpy()
        if i + 1 < b:
            if st["q"] is None:
                w[token[i + 1]] = 0
            else:
                w = np.maximum(w - st["q"][i].float().cpu().numpy(), np.float32(0))
        sums = np.cumsum(np.floor(w.astype(np.float64) * 2.0 ** UNIT).astype(np.int64))
        t = int(u_draw[s] * 2.0 ** 31) * int(sums[-1]) >> 31
        out[i] = np.searchsorted(sums, t, side="right")
        emitted[s] = i - a + 1
        lens[:, s] -= b - 1 - i
    rows = st["rows8"].cpu().numpy()
    if c["image"]:
        rows = np.minimum(rows, lens // BLOCK * BLOCK)
    return {"out": _ints(out, dev), "emitted": _ints(emitted, dev), "lens": _ints(lens, dev),
            "rows8": _ints(rows, dev)}


def _shared_exact(st):
    """Every sequence by itself: one softmax over the prefix's rows and its own."""
    c = st["case"]
    S, H, G, d, N = c["seqs"], c["kv_heads"], c["group"], c["d"], st["n"]
    dev = st["q"].device
    if N * H * G * d * (c["prefix_rows"] + c["rows"]) > 4e11:
        return None
    page = c["page"]
    block = min(BLOCK, page) if page else BLOCK
    out = torch.zeros(N, H * G, d, dtype=torch.float64, device=dev)
    lse = torch.full((N, H * G), -math.inf, dtype=torch.float64, device=dev)
    lens = {p: st[f"lens_{p}"][0].cpu().tolist() for p in ("prefix", "own")}
    held = {p: None if st[f"rows8_{p}"] is None else st[f"rows8_{p}"][0].cpu().tolist()
            for p in ("prefix", "own")}

    def rows(part, i, h, name):
        slot = torch.arange(lens[part][i][h], device=dev)
        if page:
            where = st[f"table_{part}"][i].long()[slot // page], h, slot % page
            block_at = where[0], h, slot % page // block
        else:
            where, block_at = (i, h, slot), (i, h, slot // block)
        x = st[f"{name}_{part}"][0][where].double()
        if held[part] is not None:
            m = held[part][i][h]
            y = st[f"{name}8_{part}"][0][where].double()
            y *= st[f"{name}_scale_{part}"][0][block_at].double()[:, None]
            x[:m] = y[:m]
        return x

    kept = {}
    for s in range(S):
        a, b = int(st["bounds"][s]), int(st["bounds"][s + 1])
        if a == b:
            continue
        p = int(np.searchsorted(st["groups"], s, side="right")) - 1
        p = p if s < st["groups"][-1] else -1
        for h in range(H):
            parts = {}
            for name in ("k", "v"):
                x = rows("own", s, h, name)
                if p >= 0:
                    if (p, h, name) not in kept:
                        if h == 0 and kept and next(iter(kept))[0] != p:
                            kept.clear()
                        kept[p, h, name] = rows("prefix", p, h, name)
                    x = torch.cat([kept[p, h, name], x])
                parts[name] = x
            before = lens["prefix"][p][h] if p >= 0 else 0
            own_rows = lens["own"][s][h]
            seen = torch.full((b - a,), own_rows, device=dev)
            if c["causal"]:
                seen -= torch.arange(b - a - 1, -1, -1, device=dev)
            seen = (before + seen.clamp(min=0)).repeat_interleave(G)
            q = st["q"][a:b, h * G:(h + 1) * G].double().reshape(-1, d)
            x = q @ parts["k"].T / math.sqrt(d)
            x = x.masked_fill(torch.arange(x.shape[1], device=dev) >= seen[:, None], -math.inf)
            some = seen > 0
            o = torch.zeros(x.shape[0], d, dtype=torch.float64, device=dev)
            z = torch.full((x.shape[0],), -math.inf, dtype=torch.float64, device=dev)
            if x.shape[1]:
                o[some] = torch.softmax(x[some], -1) @ parts["v"]
                z[some] = torch.logsumexp(x[some], -1)
            out[a:b, h * G:(h + 1) * G] = o.reshape(b - a, G, d)
            lse[a:b, h * G:(h + 1) * G] = z.reshape(b - a, G)
    return {"out": out, "lse": lse}
