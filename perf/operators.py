"""What is measured of the operators that fill and read the KV cache between two evictions.

One layer of a decoder that keeps its keys and values in the library's cache runs, for every
batch of new tokens, ``append`` (norm and rotate the queries and keys, write keys, values and
positions behind the rows that each slice holds) and ``attend`` (softmax attention of the new
queries over each slice's rows); between evictions ``quantize`` keeps an 8-bit image of the
full 32-row blocks, which ``attend`` then reads in place of the bf16 rows.

``run`` is one pass through one of the three, by elementary torch operations where ``own`` is
false and by the library's entry points where it is true.
"""
import math

import numpy as np
import torch

own = False

THETA = 500000.0
EPS = 1e-6
BLOCK = 32

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

#: What a case holds unless it says otherwise.
BASE = {"layers": 1, "seqs": 1, "kv_heads": 8, "group": 4, "d": 128, "dtype": "bf16", "page": 0,
        "rows": 1024, "ragged": False, "tokens": 1, "packed": False, "norm": False, "rotary": 128,
        "interleaved": False, "causal": True, "image": False, "held": 0}


def _case(name, op, **kw):
    return {"name": name, "op": op, **BASE, **kw}


def listed():
    return [
        # one decoded token of a single sequence, 32 query and 8 key heads with their norms
        _case("append_one_token", "append", rows=1638, norm=True),
        # one decoded token of each of 256 sequences in a pool of 16-row pages, the slices'
        # lengths all different after evictions; half of each head rotated, pairs side by side
        _case("append_paged_256", "append", seqs=256, page=16, rows=480, ragged=True,
              rotary=64, interleaved=True),
        # a ragged batch of prompts, straight out of one packed projection
        _case("append_prompts", "append", seqs=4, rows=513, ragged=True, tokens=8192, packed=True,
              norm=True),
        # one more full block in every slice of a 32-layer model: what a decode loop pays
        # every 32 tokens
        _case("quantize_next_block", "quantize", layers=32, rows=1696, held=1664),
        # everything that an eviction to 20 % left of two layers of 16 sequences
        _case("quantize_survivors", "quantize", layers=2, seqs=16, rows=6554),
        # a window of queries over the 512 rows of a small fp32 head
        _case("attend_window_f32", "attend", kv_heads=1, group=1, d=64, dtype="f32", rows=512,
              tokens=16),
        # one decoded token over what an eviction of 8192 rows to 20 % left
        _case("attend_one_token", "attend", rows=1638),
        # one decoded token of 64 sequences, paged, every slice with a length of its own
        _case("attend_paged_ragged", "attend", seqs=64, page=16, rows=13107, ragged=True),
        # one decoded token of 16 sequences over 32768 rows each
        _case("attend_batch16", "attend", seqs=16, rows=32768),
        # a chunk of a long prompt against everything cached before it
        _case("attend_chunk", "attend", seqs=2, rows=8704, tokens=512),
        # the 16 sequences again, from the 8-bit image
        _case("attend8_batch16", "attend", seqs=16, rows=32768, image=True),
        # a few drafted tokens of 32 sequences verified at once, from the paged 8-bit image
        _case("attend8_drafts", "attend", seqs=32, page=32, rows=13107, ragged=True, tokens=5,
              image=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "quantize", "attend", "attend", "attend8", "attend8"])
    c = dict(BASE)
    c["page"] = rng.choice([0, 0, 8, 16, 32, 64, 128])
    c["kv_heads"] = rng.choice([1, 2, 5, 8])
    c["group"] = rng.choice([1, 2, 3, 4, 6, 8])
    c["d"] = rng.choice([64, 128, 128])
    c["ragged"] = rng.random() < 0.6
    if op == "append":
        c["op"] = "append"
        c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
        c["seqs"] = _log(rng, 1, 256)
        c["rows"] = _log(rng, 1, max(1, 131072 // c["seqs"]))
        c["tokens"] = _log(rng, 1, max(1, 32768 // c["seqs"]))
        c["rotary"] = rng.choice([0, 16, c["d"] // 2, c["d"], c["d"]])
        c["interleaved"] = rng.random() < 0.4
        c["norm"] = rng.random() < 0.5
        c["packed"] = rng.random() < 0.5
    elif op == "quantize":
        c["op"] = "quantize"
        c["layers"] = _log(rng, 1, 32)
        c["seqs"] = _log(rng, 1, 32)
        most = 2 * 16 * 8 * 6554 // (c["layers"] * c["seqs"] * c["kv_heads"])
        c["rows"] = _log(rng, 1, max(1, most))
        c["held"] = rng.choice([0, 0, c["rows"] // 2 // 128 * 128])
    else:
        c["op"] = "attend"
        c["image"] = op == "attend8"
        c["dtype"] = "bf16" if c["image"] else rng.choice(["bf16", "bf16", "bf16", "f32"])
        c["seqs"] = _log(rng, 1, 64)
        c["tokens"] = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 2, 512)])
        most = 16 * 8 * 32768 // (c["seqs"] * c["kv_heads"] * (2 if c["dtype"] == "f32" else 1))
        heavy = 2 * 32 * 512 * 8704 // (c["seqs"] * c["kv_heads"] * c["group"] * c["tokens"])
        c["rows"] = _log(rng, 1, max(1, min(most, heavy, 65536)))
        c["causal"] = rng.random() < 0.8
    return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _rotary_freqs(c):
    half = c["rotary"] // 2
    return [THETA ** (-2.0 * i / c["rotary"]) for i in range(half)]


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 17)
    h = np.random.default_rng([int(seed), c["seqs"], c["rows"], c["tokens"]])
    L, S, H, G, d, dt = (c["layers"], c["seqs"], c["kv_heads"], c["group"], c["d"],
                         DTYPES[c["dtype"]])

    def normal(*shape, dtype=dt):
        return torch.empty(shape, device=dev, dtype=dtype).normal_(generator=g)

    adds = c["tokens"] if c["op"] == "append" else 0
    # rows per slice: evictions leave every slice with a length of its own
    if c["ragged"]:
        lens = h.integers(max(0, c["rows"] // 16), c["rows"] + 1, (L, S, H))
        lens.reshape(-1)[0] = c["rows"]
    else:
        lens = np.full((L, S, H), c["rows"])
    capacity = c["rows"] + adds
    if c["page"]:
        per_seq = -(-capacity // c["page"])
        capacity = per_seq * c["page"]
        pages = S * per_seq + 3
        table = torch.as_tensor(h.permutation(pages)[:S * per_seq].reshape(S, per_seq)
                                .astype(np.int32), device=dev)
        shape = (L, pages, H, c["page"])
        blocks = (L, pages, H, max(1, c["page"] // BLOCK))
    else:
        pages, per_seq, table = 0, 0, None
        shape = (L, S, H, capacity)
        blocks = (L, S, H, -(-capacity // BLOCK))
    st = {"case": c, "capacity": capacity, "pages": pages, "per_seq": per_seq, "table": table,
          "k": normal(*shape, d), "v": normal(*shape, d),
          "pos": torch.randint(0, 1 << 20, shape, generator=g, device=dev, dtype=torch.int32),
          "lens": torch.as_tensor(lens.astype(np.int32), device=dev)}
    if c["op"] == "quantize" or c["image"]:
        # heads and rows differ in size, as keys and values do
        st["k"] *= torch.exp(0.5 * normal(*shape, 1, dtype=torch.float32)).to(dt)
        st["v"] *= torch.exp(0.5 * normal(*shape, 1, dtype=torch.float32)).to(dt)
        for name in ("k", "v"):
            st[name + "8"] = torch.zeros(*shape, d, device=dev).to(torch.float8_e4m3fn) \
                if st["k"].numel() < (1 << 24) else \
                torch.zeros(*shape, d, device=dev, dtype=torch.uint8).view(torch.float8_e4m3fn)
            st[name + "_scale"] = torch.ones(blocks, device=dev)
        st["rows8"] = torch.zeros(L, S, H, dtype=torch.int32, device=dev)
    block = min(BLOCK, c["page"]) if c["page"] else BLOCK
    if c["op"] == "quantize":
        st["held"] = torch.minimum(torch.full_like(st["lens"], c["held"]),
                                   st["lens"] // block * block)
        return st
    # new tokens: n[s] of sequence s, packed behind one another
    if c["ragged"] and c["tokens"] > 1:      # by the case alone: it is what the outputs' shapes
        n = np.random.default_rng([S, c["rows"], c["tokens"]]).integers(0, c["tokens"] + 1, S)
        n[0] = c["tokens"]
    else:
        n = np.full(S, c["tokens"])
    cu = np.concatenate([[0], np.cumsum(n)])
    N = int(cu[-1])
    st["n"] = N
    st["cu"] = None if (n == c["tokens"]).all() else \
        torch.as_tensor(cu.astype(np.int32), device=dev)
    if c["op"] == "append":
        if c["packed"]:
            rows = normal(N, H * G + 2 * H, d)
            st["q"], st["nk"], st["nv"] = rows[:, :H * G], rows[:, H * G:-H], rows[:, -H:]
        else:
            st["q"], st["nk"], st["nv"] = normal(N, H * G, d), normal(N, H, d), normal(N, H, d)
        first = h.integers(c["rows"], 1 << 20, S)      # far beyond the slots after evictions
        pos = np.concatenate([first[s] + np.arange(n[s]) for s in range(S)])
        st["token_pos"] = torch.as_tensor(pos.astype(np.int32), device=dev)
        st["lens_in"] = st["lens"][0].clone()
        st["q_out"] = torch.empty(N, H * G, d, device=dev, dtype=dt)
        st["freqs"] = torch.tensor(_rotary_freqs(c), dtype=torch.float64, device=dev)
        for name in ("q_norm", "k_norm"):
            st[name] = (1 + 0.2 * normal(d, dtype=torch.float32)).to(dt) if c["norm"] else None
        return st
    # queries that look for one of the slice's rows each, next to everything else
    st["q"] = normal(N, H * G, d)
    seq = torch.as_tensor(np.repeat(np.arange(S), n), device=dev)
    ln = st["lens"][0][seq].clamp(min=1).float()                               # [N, H]
    aim = (torch.rand(N, H, generator=g, device=dev) * ln).long()
    hub = _at(st, "k", seq[:, None].expand(N, H), torch.arange(H, device=dev).expand(N, H),
              aim).float()
    hub = 6 * hub / hub.norm(dim=-1, keepdim=True)
    st["q"] += hub.repeat_interleave(G, dim=1).to(dt)
    st["out"] = torch.empty(N, H * G, d, device=dev, dtype=dt)
    st["lse"] = torch.empty(N, H * G, device=dev)
    if c["image"]:
        st["held"] = torch.zeros_like(st["lens"])
        _quantize_plain(st)
    return st


def _at(st, name, s, h, slot):
    """Rows of layer 0 at (sequence, head, slot), tensors of one shape."""
    t, page = st[name][0], st["case"]["page"]
    if page:
        return t[st["table"].long()[s, slot // page], h, slot % page]
    return t[s, h, slot]


def _whole(st, name, layer=0):
    """[seqs, kv_heads, capacity, ...] of one layer, pages in order."""
    t, page = st[name][layer], st["case"]["page"]
    if not page:
        return t
    t = t[st["table"].long()]                            # [S, pages, H, page, ...]
    t = t.transpose(1, 2)
    return t.reshape(*t.shape[:2], -1, *t.shape[4:])


# ---------------------------------------------------------------------------
# The operators
# ---------------------------------------------------------------------------

def _handle(st):
    """The objects that a user's program makes once for its buffers."""
    if "handle" not in st:
        from streaming_kv_cache_step_gb300 import nexus
        c = st["case"]
        cache = nexus.Cache(k=st["k"], v=st["v"], pos=st["pos"], lens=st["lens"],
                            layers=c["layers"], seqs=c["seqs"], kv_heads=c["kv_heads"],
                            group=c["group"], head_dim=c["d"], capacity=st["capacity"],
                            page_size=c["page"], num_pages=st["pages"],
                            max_pages_per_seq=st["per_seq"], block_table=st["table"])
        image = rotary = ws = None
        if "k8" in st:
            image = nexus.Image(k=st["k8"], v=st["v8"], k_scale=st["k_scale"],
                                v_scale=st["v_scale"], rows=st["rows8"])
        if c["op"] == "append" and c["rotary"]:
            rotary = nexus.Rotary(_rotary_freqs(c), interleaved=c["interleaved"],
                                  device=st["k"].device)
        if c["op"] == "attend":
            ws = nexus.alloc_attend_workspace(cache, tokens=st["n"], max_tokens=c["tokens"])
        st["handle"] = nexus, cache, image, rotary, ws, nexus.new_status(st["k"].device)
    return st["handle"]


def run(state):
    st, c = state, state["case"]
    if own:
        nexus, cache, image, rotary, ws, status = _handle(st)
        if c["op"] == "append":
            nexus.append(cache, 0, st["q"], st["nk"], st["nv"], st["token_pos"], st["q_out"],
                         status, max_tokens=c["tokens"], cu_tokens=st["cu"],
                         lens_in=st["lens_in"], rotary=rotary, q_norm=st["q_norm"],
                         k_norm=st["k_norm"], eps=EPS)
        elif c["op"] == "quantize":
            nexus.quantize(cache, image, status, rows_in=st["held"])
        else:
            nexus.attend(cache, 0, st["q"], st["out"], ws, status, max_tokens=c["tokens"],
                         cu_tokens=st["cu"], causal=c["causal"], lse=st["lse"], image=image)
    elif c["op"] == "append":
        _append_plain(st)
    elif c["op"] == "quantize":
        _quantize_plain(st)
    else:
        _attend_plain(st)
    if c["op"] == "append":
        return {"q": st["q_out"], "k": st["k"], "v": st["v"], "pos": st["pos"],
                "lens": st["lens"]}
    if c["op"] == "quantize":
        return {"k8": st["k8"], "v8": st["v8"], "k_scale": st["k_scale"],
                "v_scale": st["v_scale"], "rows": st["rows8"]}
    return {"out": st["out"], "lse": st["lse"]}


def _cu(st):
    c = st["case"]
    if st["cu"] is not None:
        return st["cu"].long()
    return torch.arange(c["seqs"] + 1, device=st["k"].device) * c["tokens"]


def _rotate(x, pos, c, freqs):
    r = c["rotary"]
    if not r:
        return x
    ang = pos.double()[:, None] * freqs
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
    head, rest = x[..., :r], x[..., r:]
    if c["interleaved"]:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = head[..., :r // 2], head[..., r // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, rest], -1)


def _normed(x, weight):
    x = x.float()
    if weight is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()


def _append_plain(st):
    c, dt = st["case"], st["k"].dtype
    S, H, N = c["seqs"], c["kv_heads"], st["n"]
    cu = _cu(st)
    tok = torch.arange(N, device=cu.device)
    seq = torch.searchsorted(cu, tok, right=True) - 1
    st["q_out"].copy_(_rotate(_normed(st["q"], st["q_norm"]), st["token_pos"], c, st["freqs"]))
    rows_k = _rotate(_normed(st["nk"], st["k_norm"]), st["token_pos"], c, st["freqs"]).to(dt)
    slot = st["lens_in"].long()[seq] + (tok - cu[seq])[:, None]                     # [N, H]
    head = torch.arange(H, device=cu.device).expand(N, H)
    if c["page"]:
        where = st["table"].long()[seq[:, None], slot // c["page"]], head, slot % c["page"]
    else:
        where = seq[:, None].expand(N, H), head, slot
    st["k"][0].index_put_(where, rows_k)
    st["v"][0].index_put_(where, st["nv"].to(dt))
    st["pos"][0].index_put_(where, st["token_pos"][:, None].expand(N, H))
    st["lens"][0] = st["lens_in"] + (cu[1:] - cu[:-1]).int()[:, None]


def _quantize_plain(st):
    """Blocks [held / b, lens / b) of every slice: the power of two that brings the block's
    largest value to at most 448, and the rows over it in e4m3."""
    c, page = st["case"], st["case"]["page"]
    b = min(BLOCK, page) if page else BLOCK
    L, S, H, d = c["layers"], c["seqs"], c["kv_heads"], c["d"]
    per = st["capacity"] // b                      # full blocks that a slice can hold
    t = torch.arange(per, device=st["k"].device)
    pick = (t >= (st["held"] // b)[..., None]) & (t < (st["lens"] // b)[..., None])
    l, s, h, t = pick.nonzero(as_tuple=True)
    row = torch.arange(b, device=t.device)
    if page:
        p = st["table"].long()[s, t * b // page]
        where = l[:, None], p[:, None], h[:, None], (t * b % page)[:, None] + row
        at = l, p, h, t * b % page // b
    else:
        where = l[:, None], s[:, None], h[:, None], (t * b)[:, None] + row
        at = l, s, h, t
    for name in ("k", "v"):
        x = st[name][where].float()
        most = x.abs().amax((1, 2))
        m, e = torch.frexp(most)                   # most = m 2^e, m in [0.5, 1)
        e = torch.where(m > 0.875, e - 8, e - 9)
        scale = torch.where(most > 0, torch.ldexp(torch.ones_like(most), e.clamp(-100, 120)), 1.0)
        codes = (x / scale[:, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        st[name + "8"].view(torch.uint8)[where] = codes.view(torch.uint8)
        st[name + "_scale"][at] = scale
    st["rows8"].copy_(st["lens"] // b * b)


def _keys_and_values(st):
    """[seqs, kv_heads, capacity, d] in 32 bits: the image's rows where it holds them."""
    c = st["case"]
    got = []
    for name in ("k", "v"):
        x = _whole(st, name).float()
        if c["image"]:
            b = min(BLOCK, c["page"]) if c["page"] else BLOCK
            codes = _whole(st, name + "8").float()
            scale = _whole(st, name + "_scale").repeat_interleave(b, dim=2)[:, :, :x.shape[2]]
            held = torch.arange(x.shape[2], device=x.device) < st["rows8"][0][..., None]
            x = torch.where(held[..., None], codes * scale[..., None], x)
        got.append(x)
    return got


def _attend_plain(st):
    c = st["case"]
    S, H, G, d, M = c["seqs"], c["kv_heads"], c["group"], c["d"], c["tokens"]
    dev = st["k"].device
    k, v = _keys_and_values(st)
    T = k.shape[2]
    cu = _cu(st)
    n = cu[1:] - cu[:-1]
    i = torch.arange(M, device=dev)
    here = i < n[:, None]                                                      # [S, M]
    tok = (cu[:-1, None] + i).clamp(max=max(0, st["n"] - 1))
    q = st["q"].float()[tok].reshape(S, M, H, G, d).permute(0, 2, 1, 3, 4).reshape(S, H, M * G, d)
    x = torch.matmul(q, k.transpose(-1, -2)) * (1 / math.sqrt(d))
    lens = st["lens"][0].long()
    last = (n[:, None] - 1 - i) if c["causal"] else torch.zeros_like(here, dtype=torch.long)
    limit = (lens[:, :, None] - last[:, None]).clamp(min=0).repeat_interleave(G, dim=2)
    off = torch.arange(T, device=dev) >= limit[..., None]
    x.masked_fill_(off, -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top > -math.inf, top, 0.0))
    z = e.sum(-1, keepdim=True)
    lse = (top + torch.log(z))[..., 0]
    v = v.masked_fill((torch.arange(T, device=dev) >= lens[..., None])[..., None], 0)
    o = torch.matmul(e, v) / torch.where(z > 0, z, 1.0)
    o = o.reshape(S, H, M, G, d).permute(0, 2, 1, 3, 4).reshape(S, M, H * G, d)
    lse = lse.reshape(S, H, M, G).permute(0, 2, 1, 3).reshape(S, M, H * G)
    st["out"].copy_(o[here])
    st["lse"].copy_(lse[here])


# ---------------------------------------------------------------------------
# What a pass cannot do without, and the definition in 64 bits
# ---------------------------------------------------------------------------

def _mean_rows(c):
    return (c["rows"] + c["rows"] // 16) / 2 if c["ragged"] else c["rows"]


def _mean_tokens(c):
    if c["ragged"] and c["tokens"] > 1:
        return c["tokens"] + (c["seqs"] - 1) * c["tokens"] / 2
    return c["seqs"] * c["tokens"]


def work(case):
    c = case
    S, H, G, d, size = c["seqs"], c["kv_heads"], c["group"], c["d"], 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "append":
        rows = _mean_tokens(c) * (G + 2) * H
        return {"bytes": rows * d * size * 2 + _mean_tokens(c) * (4 + 4 * H),
                "flops": rows * d * 6}
    if c["op"] == "quantize":
        rows = c["layers"] * S * H * max(0, _mean_rows(c) - c["held"])
        return {"bytes": 2 * rows * (d * 3 + 4 / BLOCK), "flops": 2 * rows * d * 2}
    rows = S * H * _mean_rows(c)
    if c["image"]:
        size_kv = 1 + 4 / BLOCK / d
    else:
        size_kv = size
    tokens = _mean_tokens(c)
    return {"bytes": 2 * rows * d * size_kv + tokens * H * G * (2 * d * size + 4),
            "flops": 4 * d * rows * G * tokens / S}


def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _append_exact, "quantize": _quantize_exact, "attend": _attend_exact}[
        case["op"]](st)


def _bounds(st):
    return [int(x) for x in _cu(st).cpu()]


def _append_exact(st):
    c, cu = st["case"], _bounds(st)
    H, d, r = c["kv_heads"], c["d"], c["rotary"]
    new = {}
    for name, weight in (("q", st["q_norm"]), ("nk", st["k_norm"])):
        x = st[name].double()
        if weight is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS) * weight.double()
        if r:
            phase = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                                st["token_pos"].double()[:, None] * st["freqs"])[:, None, :]
            i = torch.arange(r // 2, device=x.device)
            first, second = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + r // 2)
            z = torch.complex(x[..., first], x[..., second]) * phase
            x[..., first], x[..., second] = z.real, z.imag
        new[name] = x
    k, v, pos, lens = st["k"].double(), st["v"].double(), st["pos"].clone(), st["lens"].clone()
    heads = torch.arange(H, device=k.device)
    for s in range(c["seqs"]):
        a, b = cu[s], cu[s + 1]
        slot = st["lens_in"][s].long()[None] + torch.arange(b - a, device=k.device)[:, None]
        if c["page"]:
            at = 0, st["table"][s].long()[slot // c["page"]], heads[None], slot % c["page"]
        else:
            at = 0, s, heads[None], slot
        k[at], v[at] = new["nk"][a:b], st["nv"][a:b].double()
        pos[at] = st["token_pos"][a:b, None].expand(b - a, H)
        lens[0, s] = st["lens_in"][s] + (b - a)
    return {"q": new["q"], "k": k, "v": v, "pos": pos, "lens": lens}


def _quantize_exact(st):
    c, page = st["case"], st["case"]["page"]
    b = min(BLOCK, page) if page else BLOCK
    got = {"rows": st["lens"] // b * b}
    for name in ("k", "v"):
        codes, scales = st[name + "8"].double(), st[name + "_scale"].double()
        for l in range(c["layers"]):
            x = _whole(st, name, l).double()                              # [S, H, capacity, d]
            full = x.shape[2] // b
            x = x[:, :, :full * b].unflatten(2, (full, b))
            m, e = torch.frexp(x.abs().amax((3, 4)) / 448)                # in [2^(e - 1), 2^e)
            e = torch.where(m == 0.5, e - 1, e).clamp(-100, 120)
            scale = torch.where(m > 0, torch.exp2(e.double()), 1.0)
            y = x / scale[..., None, None]
            # e4m3 has steps of 2^-3 within a power of two, and of 2^-9 below 2^-6
            step = torch.exp2((torch.frexp(y)[1] - 1).clamp(min=-6).double() - 3)
            y = torch.round(y / step) * step
            at = torch.arange(full, device=x.device)
            new = (at >= st["held"][l][..., None] // b) & (at < st["lens"][l][..., None] // b)
            s, h, t = new.nonzero(as_tuple=True)
            row = (t * b)[:, None] + torch.arange(b, device=t.device)
            if page:
                p = st["table"].long()[s, t * b // page]
                codes[l][p[:, None], h[:, None], row % page] = y[s, h, t]
                scales[l][p, h, t * b % page // b] = scale[s, h, t]
            else:
                codes[l][s[:, None], h[:, None], row] = y[s, h, t]
                scales[l][s, h, t] = scale[s, h, t]
        got[name + "8"], got[name + "_scale"] = codes, scales
    return got


def _attend_exact(st):
    c, cu = st["case"], _bounds(st)
    H, G, d = c["kv_heads"], c["group"], c["d"]
    out = torch.zeros(st["n"], H * G, d, dtype=torch.float64, device=st["k"].device)
    lse = torch.full((st["n"], H * G), -math.inf, dtype=torch.float64, device=out.device)
    if st["n"] * H * G * d * c["rows"] > 1e11:
        return None
    b = min(BLOCK, c["page"]) if c["page"] else BLOCK
    lens = st["lens"][0].cpu().tolist()
    held = st["rows8"][0].cpu().tolist() if c["image"] else None
    heads = torch.arange(H, device=out.device)
    for s in range(c["seqs"]):
        most, n = max(lens[s]), cu[s + 1] - cu[s]
        if not most or not n:
            continue
        slot = torch.arange(most, device=out.device)
        if c["page"]:
            p = st["table"][s].long()[slot // c["page"]]
            at = p[None], heads[:, None], (slot % c["page"])[None]
            at_block = p[None], heads[:, None], (slot % c["page"] // b)[None]
        else:
            at = s, heads[:, None], slot[None]
            at_block = s, heads[:, None], (slot // b)[None]
        rows = {}
        for name in ("k", "v"):
            x = st[name][0][at].double()
            if c["image"]:
                y = st[name + "8"][0][at].double() * st[name + "_scale"][0][at_block].double()[..., None]
                x = torch.where((slot[None] < torch.tensor(held[s], device=slot.device)[:, None])[..., None], y, x)
            rows[name] = x
        q = st["q"][cu[s]:cu[s + 1]].double().reshape(n, H, G, d)
        for h in range(H):
            x = q[:, h].reshape(n * G, d) @ rows["k"][h].T / math.sqrt(d)
            seen = torch.full((n,), lens[s][h], device=slot.device)
            if c["causal"]:
                seen = seen - torch.arange(n - 1, -1, -1, device=slot.device)
            seen = seen.repeat_interleave(G)
            x = x.masked_fill(slot[None] >= seen[:, None], -math.inf)
            some = seen > 0
            w = torch.softmax(x[some], -1)
            o = torch.zeros(n * G, d, dtype=torch.float64, device=slot.device)
            o[some] = w @ rows["v"][h]
            out[cu[s]:cu[s + 1], h * G:(h + 1) * G] = o.reshape(n, G, d)
            z = torch.full((n * G,), -math.inf, dtype=torch.float64, device=slot.device)
            z[some] = torch.logsumexp(x[some], -1)
            lse[cu[s]:cu[s + 1], h * G:(h + 1) * G] = z.reshape(n, G)
    return {"out": out, "lse": lse}
