"""Cases of the cache operators around the tree: rotary positions written into a
cache, attention of one new token per sequence over a batch of caches, and the
page bookkeeping of a paged cache. `own` selects the library's calls; otherwise
`run` computes the same in elementary torch operations."""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ELT = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # One short conversation of the small fp32 configuration: a call whose launch is what it costs.
        {"name": "attend one short", "op": "attend", "seqs": 1, "kv": 1, "group": 4, "d": 64, "chunk": 16, "tokens": 203, "cache": "f32", "q": "f32", "paged": True},
        # One request at the full million-token context, dense: the other arm of the routed decode step.
        {"name": "attend 1M context", "op": "attend", "seqs": 1, "kv": 4, "group": 8, "d": 128, "chunk": 64, "tokens": 1048576 + 37, "cache": "bf16", "q": "f32", "paged": True},
        # A serving batch of medium contexts with bf16 queries, ragged up to 32K.
        {"name": "attend 8 x 32K", "op": "attend", "seqs": 8, "kv": 8, "group": 4, "d": 128, "chunk": 64, "tokens": 32768, "cache": "bf16", "q": "bf16", "paged": True},
        # Many short conversations at once, pages of 16, some slots empty.
        {"name": "attend 160 ragged", "op": "attend", "seqs": 160, "kv": 4, "group": 4, "d": 128, "chunk": 16, "tokens": 3001, "cache": "bf16", "q": "f32", "paged": True},
        # One decode step of four requests: four tokens' projections into their pages.
        {"name": "append 4 tokens", "op": "append", "new": 4, "seqs": 4, "kv": 4, "group": 8, "d": 128, "chunk": 64, "pairs": 64, "layout": "interleaved", "scaling": "none", "src": "bf16", "cache": "bf16", "q": "f32", "paged": True, "far": 1000000},
        # A prompt chunk: the half layout on part of the head, scaled for a long context.
        {"name": "append 16K prompt", "op": "append", "new": 16384, "seqs": 3, "kv": 8, "group": 4, "d": 128, "chunk": 64, "pairs": 48, "layout": "half", "scaling": "yarn", "src": "bf16", "cache": "bf16", "q": "bf16", "paged": True, "far": 120000},
        # The gradient of rotated fp32 queries of a short batch, odd pair count.
        {"name": "turn back 257", "op": "apply", "new": 257, "heads": 4, "d": 64, "pairs": 13, "layout": "interleaved", "scaling": "linear", "src": "f32", "out": "f32", "inverse": True, "far": 5000},
        # Keys of a long prompt turned in bf16, bands scaling.
        {"name": "turn 32K keys", "op": "apply", "new": 32768, "heads": 32, "d": 128, "pairs": 64, "layout": "half", "scaling": "bands", "src": "bf16", "out": "bf16", "inverse": False, "far": 262144},
        # One step of a small beam: old beams freed, new ones forked, all made longer.
        {"name": "beam step of 4", "op": "beam", "slots": 8, "forks": 4, "kv": 1, "d": 64, "chunk": 16, "tokens": 300, "grow": 1, "cache": "f32"},
        # Parallel sampling over a large pool: 48 forks, every sequence longer by a speculated block.
        {"name": "fork 48 of 128", "op": "beam", "slots": 128, "forks": 48, "kv": 8, "d": 128, "chunk": 64, "tokens": 4096, "grow": 70, "cache": "bf16"},
        # A small pool packed after a few requests ended.
        {"name": "compact 512 pages", "op": "compact", "slots": 6, "kv": 1, "d": 64, "chunk": 16, "tokens": 900, "cache": "f32", "live": 0.5},
        # A large fragmented pool packed.
        {"name": "compact 32K pages", "op": "compact", "slots": 40, "kv": 8, "d": 128, "chunk": 64, "tokens": 6000, "cache": "bf16", "live": 0.6},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "apply", "beam", "compact"])
    d = rng.choice([64, 128, 128])
    chunk = rng.choice([4, 16, 64, 64, rng.randint(2, 128)])
    cache = rng.choice(["bf16", "bf16", "f32"])
    kv = rng.choice([1, 2, 4, 8])
    pairs = rng.choice([d // 2, d // 4, rng.randint(1, d // 2)])
    layout = rng.choice(["interleaved", "half"])
    scaling = rng.choice(["none", "linear", "ntk", "yarn", "bands"])
    far = _log(rng, 100, 4000000)
    if op == "attend":
        seqs = _log(rng, 1, 256)
        most = (1 << 28) // (seqs * kv * d)
        return {"op": op, "seqs": seqs, "kv": kv, "group": rng.choice([1, 2, 3, 4, 5, 7, 8, 8, 12, 16]), "d": d, "chunk": chunk, "tokens": _log(rng, 1, max(1, min(most, 600000))), "cache": cache, "q": rng.choice(["f32", "bf16"]), "paged": rng.random() < 0.8}
    if op == "append":
        return {"op": op, "new": _log(rng, 1, 8192), "seqs": rng.choice([1, 2, 5, 16]), "kv": kv, "group": rng.choice([1, 2, 4, 8]) if kv < 8 else rng.choice([1, 2, 4]), "d": d, "chunk": chunk, "pairs": pairs, "layout": layout, "scaling": scaling, "src": rng.choice(["bf16", "f32"]), "cache": cache, "q": rng.choice(["f32", "bf16"]), "paged": rng.random() < 0.8, "far": far}
    if op == "apply":
        return {"op": op, "new": _log(rng, 1, 20000), "heads": rng.choice([1, 3, 4, 8, 16, 32]), "d": d, "pairs": pairs, "layout": layout, "scaling": scaling, "src": rng.choice(["bf16", "f32"]), "out": rng.choice(["bf16", "f32"]), "inverse": rng.random() < 0.5, "far": far}
    slots = _log(rng, 3, 64)
    tokens = _log(rng, 1, max(2, min(8000, (1 << 28) // (slots * kv * d))))
    if op == "beam":
        return {"op": op, "slots": slots, "forks": rng.randint(1, max(1, slots // 2)), "kv": kv, "d": d, "chunk": chunk, "tokens": tokens, "grow": rng.choice([1, 1, rng.randint(1, 200)]), "cache": cache}
    return {"op": op, "slots": slots, "kv": kv, "d": d, "chunk": chunk, "tokens": tokens, "cache": cache, "live": rng.uniform(0.2, 0.95)}


def _rope_args(c):
    """The rotation of a case: base 10000, and what its scaling needs."""
    a = {"head_dim": c["d"], "pairs": c["pairs"], "layout": c["layout"], "base": 10000.0, "scaling": c["scaling"]}
    if c["scaling"] != "none":
        a["factor"] = 8.0
    if c["scaling"] == "yarn":
        a.update(original_tokens=16384.0, low=1.0, high=32.0)
    if c["scaling"] == "bands":
        a.update(original_tokens=8192.0, low=1.0, high=4.0)
    return a


def _own_rope(c):
    """The case's rotation as the library is asked for it. The forms in this file end a yarn ramp at
    the last pair at the latest, the library at freq_dim - 1 = 2 pairs - 1. Where x(low) lies beyond the
    last pair (6 pairs or fewer here), a `low` whose x is just below it asks for the same ramp."""
    a = _rope_args(c)
    if c["scaling"] == "yarn" and c["pairs"] > 1:
        last = a["original_tokens"] / (2 * math.pi) * a["base"] ** (-(c["pairs"] - 1.02) / c["pairs"])
        a["low"] = max(a["low"], last)
    return _lib().Rope(**a)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, device="cuda", generator=g) * scale).to(dtype)


def _pool(g, n, c, dtype):
    """[n, C, d] of normal values, made in pieces so that the fp32 draw stays small."""
    out = torch.empty(n, c["chunk"], c["d"], dtype=dtype, device="cuda")
    step = max(1, (1 << 26) // (c["chunk"] * c["d"]))
    for i in range(0, n, step):
        out[i:i + step] = torch.randn(out[i:i + step].shape, device="cuda", generator=g)
    return out


def _lib():
    from hierarchical_sparse_attention_zha_b200 import zha
    return zha


def _config(c, hq):
    return _lib().make_config(c["kv"], hq, c["d"], c["chunk"], 1, 1, DTYPES[c["cache"]], 1 << 30)


def _spread(seqs, tokens):
    """Ragged lengths up to `tokens`, every twentieth slot empty; their order is the seed's."""
    n = [tokens * (i + 1) // seqs for i in range(seqs)]
    return [0 if i % 20 == 7 and i < seqs - 1 else n[i] for i in range(seqs)]


def _lengths(r, seqs, tokens):
    return r.permutation(np.array(_spread(seqs, tokens), np.int64))


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = np.random.default_rng(seed)
    s = {"case": c}
    if c["op"] == "attend":
        S, H, G, d, C = c["seqs"], c["kv"], c["group"], c["d"], c["chunk"]
        dt = DTYPES[c["cache"]]
        blocks = -(-c["tokens"] // C)
        if c["paged"]:
            pages = S * H * blocks + 5
            s["K"], s["V"] = _pool(g, pages, c, dt), _pool(g, pages, c, dt)
            s["table"] = torch.randperm(pages, device="cuda", generator=g)[: S * H * blocks].to(torch.int32).reshape(S, H, blocks)
        else:
            ld = blocks * C + 3
            s["K"] = torch.empty(S, H, ld, d, dtype=dt, device="cuda")
            s["V"] = torch.empty(S, H, ld, d, dtype=dt, device="cuda")
            for x in (s["K"], s["V"]):
                for i in range(S):
                    x[i] = torch.randn(H, ld, d, device="cuda", generator=g)
            s["table"] = None
        s["Q"] = _randn(g, (S, H * G, d), DTYPES[c["q"]], 2.0)
        s["n"] = torch.from_numpy(_lengths(r, S, c["tokens"])).cuda()
        if own:
            zha = _lib()
            s["cfg"] = _config(c, H * G)
            s["kvc"] = zha.kv_batch(s["K"], s["V"], s["table"])
            s["ws"] = torch.empty(max(1, zha.attend_batch_workspace_bytes(s["cfg"], S, c["tokens"])), dtype=torch.uint8, device="cuda")
            s["out"] = torch.empty(S, H * G, d, dtype=DTYPES[c["q"]], device="cuda")
            s["lse"] = torch.empty(S, H * G, device="cuda")
    elif c["op"] == "append":
        S, H, T, C, d = c["seqs"], c["kv"], c["new"], c["chunk"], c["d"]
        hq = H * c["group"]
        dt = DTYPES[c["cache"]]
        # a fused projection's rows: queries, keys and values side by side
        s["qkv"] = _randn(g, (T, hq + 2 * H, d), DTYPES[c["src"]])
        seq = r.permutation(np.arange(T) % S)
        start = r.integers(0, 3 * C, S)
        order = np.argsort(seq, kind="stable")
        first = np.searchsorted(seq[order], seq[order])
        index = np.empty(T, np.int64)
        index[order] = start[seq[order]] + np.arange(T) - first
        blocks = 3 + -(-(-(-T // S)) // C)
        if c["paged"]:
            pages = S * H * blocks + 3
            s["table"] = torch.randperm(pages, device="cuda", generator=g)[: S * H * blocks].to(torch.int32).reshape(S, H, blocks)
            shape = (pages, C, d)
        else:
            s["table"] = None
            shape = (S, H, blocks * C, d)
        s["K"] = torch.zeros(shape, dtype=dt, device="cuda")
        s["V"] = torch.zeros(shape, dtype=dt, device="cuda")
        s["seq"] = torch.from_numpy(seq.astype(np.int32)).cuda()
        s["index"] = torch.from_numpy(index).cuda()
        s["pos"] = s["index"] + int(r.integers(0, c["far"] + 1))
        if own:
            zha = _lib()
            s["cfg"] = _config(c, hq)
            s["rope"] = _own_rope(c)
            s["kvc"] = zha.kv_batch(s["K"], s["V"], s["table"])
            s["out"] = torch.empty(T, hq, d, dtype=DTYPES[c["q"]], device="cuda")
    elif c["op"] == "apply":
        s["X"] = _randn(g, (c["new"], c["heads"], c["d"]), DTYPES[c["src"]])
        s["pos"] = torch.from_numpy(r.integers(0, c["far"] + 1, c["new"])).cuda()
        if own:
            s["rope"] = _own_rope(c)
            s["out"] = torch.empty(c["new"], c["heads"], c["d"], dtype=DTYPES[c["out"]], device="cuda")
    else:
        s.update(_pages_state(c, r, g))
        if own:
            zha = _lib()
            s["cfg"] = _config(c, c["kv"])
            s["pool"] = zha.page_pool(s["K"], s["V"], s["table"], s["refs"])
            s["ws"] = torch.empty(zha.pages_workspace_bytes(s["cfg"], s["pool"], c["slots"]), dtype=torch.uint8, device="cuda")
    return s


def _pages_layout(c):
    blocks = -(-(c["tokens"] + c.get("grow", 0)) // c["chunk"])
    return blocks, c["slots"] * c["kv"] * blocks + 8


def _pages_state(c, r, g):
    """A pool in use: sequences of ragged lengths in shuffled pages, some sharing
    their first blocks with another, some slots empty. The table and the counts
    lie in one buffer, with a copy that each pass starts from."""
    S, H, C = c["slots"], c["kv"], c["chunk"]
    blocks, pages = _pages_layout(c)
    n = _lengths(r, S, c["tokens"])
    n[n == 0] = 1 if c["op"] == "beam" else 0
    if c["op"] == "compact":
        n[r.random(S) > c["live"] + 0.3] = 0
        n = np.minimum(n, np.maximum(1, (n * min(1.0, 2 * c["live"])).astype(np.int64)) * (n > 0))
        n[0] = max(1, n[0])
    used = -(-n // C)
    table = np.full((S, H, blocks), -1, np.int64)
    have = np.arange(blocks)[None, None, :] < used[:, None, None]
    have = np.broadcast_to(have, table.shape)
    table[have] = r.permutation(pages)[: int(have.sum())]
    for i in range(2, S, 5):      # the first blocks shared with the slot before
        share = int(min(n[i], n[i - 1]) // C // 2)
        table[i, :, :share] = table[i - 1, :, :share]
    refs = np.bincount(table[table >= 0], minlength=pages)
    cells = -(-table.size // 4) * 4
    book = np.zeros(cells + pages, np.int32)
    book[: table.size] = table.reshape(-1)
    book[cells:] = refs
    book0 = torch.from_numpy(book).cuda()
    book = book0.clone()
    s = {"book0": book0, "book": book, "table": book[: table.size].view(S, H, blocks), "refs": book[cells:],
         "K": _pool(g, pages, c, DTYPES[c["cache"]]), "V": _pool(g, pages, c, DTYPES[c["cache"]])}
    if c["op"] == "beam":
        pick = r.permutation(S)
        dst = np.sort(pick[: c["forks"]])
        src = r.choice(np.sort(pick[c["forks"]:]), c["forks"])
        now = n.copy()
        now[dst] = n[src]
        s["src"] = torch.from_numpy(src.astype(np.int32)).cuda()
        s["dst"] = torch.from_numpy(dst.astype(np.int32)).cuda()
        s["fork_n"] = torch.from_numpy(n[src]).cuda()
        s["all"] = torch.arange(S, dtype=torch.int32, device="cuda")
        s["new_n"] = torch.from_numpy(now + c["grow"]).cuda()
    else:
        s["map"] = torch.empty(pages, dtype=torch.int32, device="cuda")
        s["live"] = torch.empty(1, dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    return {"attend": _attend, "append": _append, "apply": _apply, "beam": _beam, "compact": _compact}[s["case"]["op"]](s)


def _attend(s):
    c = s["case"]
    S, H, G, d, C, N = c["seqs"], c["kv"], c["group"], c["d"], c["chunk"], c["tokens"]
    if own:
        return _lib().attend_batch_kv(s["cfg"], s["Q"], s["kvc"], S, s["n"], N, out=s["out"], lse=s["lse"], ws=s["ws"])
    if s["table"] is None:
        K, V = s["K"][:, :, :N], s["V"][:, :, :N]
    else:
        at = s["table"].long()
        K, V = (x[at].reshape(S, H, -1, d)[:, :, :N] for x in (s["K"], s["V"]))
    seen = (torch.arange(N, device="cuda")[None] < s["n"][:, None])[:, None, None]
    q = s["Q"].float().reshape(S, H, G, d) / math.sqrt(d)
    x = torch.matmul(q, K.float().transpose(-1, -2)).masked_fill(~seen, -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, V.float()) / total.clamp(min=1e-30)
    lse = (top + torch.log(total)).masked_fill(total == 0, -math.inf)
    return o.reshape(S, H * G, d).to(s["Q"].dtype), lse.reshape(S, H * G)


def _angles(c):
    """Angle per position of each pair, in 64 bits, and the amplitude."""
    a = _rope_args(c)
    i = torch.arange(a["pairs"], dtype=torch.float64, device="cuda")
    dim, base, f, amp = 2 * a["pairs"], a["base"], a.get("factor", 1.0), 1.0
    if a["scaling"] == "ntk" and dim > 2:
        base = base * f ** (dim / (dim - 2))
    theta = base ** (-2 * i / dim)
    if a["scaling"] == "linear" or (a["scaling"] == "ntk" and dim == 2):
        theta = theta / f
    elif a["scaling"] == "yarn":
        def where(turns):
            return dim * math.log(a["original_tokens"] / (2 * math.pi * turns)) / (2 * math.log(base))
        lo, hi = max(math.floor(where(a["high"])), 0), min(math.ceil(where(a["low"])), a["pairs"] - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        theta = theta * (1 - ramp) + theta / f * ramp
        amp = 0.1 * math.log(f) + 1
    elif a["scaling"] == "bands":
        turns = a["original_tokens"] * theta / (2 * math.pi)
        keep = ((turns - a["low"]) / (a["high"] - a["low"])).clamp(0, 1)
        theta = keep * theta + (1 - keep) * theta / f
    return theta, amp


def _turned(c, x, pos, back=False):
    """x [T, heads, d] in fp32, turned at its positions (or back: the transpose)."""
    theta, amp = _angles(c)
    P = c["pairs"]
    phi = pos.double()[:, None] * theta
    cos, sin = (amp * torch.cos(phi)).float()[:, None], (amp * torch.sin(phi)).float()[:, None]
    if back:
        sin = -sin
    if c["layout"] == "half":
        a, b = x[..., :P], x[..., P:2 * P]
    else:
        a, b = x[..., 0:2 * P:2], x[..., 1:2 * P:2]
    u, v = a * cos - b * sin, a * sin + b * cos
    y = torch.cat((u, v), -1) if c["layout"] == "half" else torch.stack((u, v), -1).flatten(-2)
    return torch.cat((y, x[..., 2 * P:]), -1)


def _append(s):
    c = s["case"]
    H, C = c["kv"], c["chunk"]
    hq = H * c["group"]
    q, k, v = s["qkv"][:, :hq], s["qkv"][:, hq:hq + H], s["qkv"][:, hq + H:]
    if own:
        out = _lib().rope_append_kv(s["cfg"], s["rope"], q, k, v, s["kvc"], c["seqs"], s["seq"], s["index"], s["pos"], q_out=s["out"])
        return out, s["K"], s["V"]
    seq, head = s["seq"].long()[:, None], torch.arange(H, device="cuda")[None]
    at = s["index"][:, None]
    if s["table"] is None:
        where = (seq, head, at)
    else:
        where = (s["table"][seq, head, at // C].long(), at % C)
    s["K"][where] = _turned(c, k.float(), s["pos"]).to(s["K"].dtype)
    s["V"][where] = v.to(s["V"].dtype)
    return _turned(c, q.float(), s["pos"]).to(DTYPES[c["q"]]), s["K"], s["V"]


def _apply(s):
    c = s["case"]
    if own:
        return _lib().rope_apply(s["rope"], s["X"], s["pos"], out=s["out"], inverse=c["inverse"])
    return _turned(c, s["X"].float(), s["pos"], c["inverse"]).to(DTYPES[c["out"]])


def _take(refs, want):
    """The lowest free pages, one for each true entry of `want` in order (-1 elsewhere)."""
    free = torch.nonzero(refs == 0).flatten()
    rank = (torch.cumsum(want.flatten(), 0) - 1).clamp(min=0).reshape(want.shape)
    return torch.where(want, free[rank.clamp(max=free.numel() - 1)], -1)


def _beam(s):
    c = s["case"]
    C, table, refs = c["chunk"], s["table"], s["refs"]
    s["book"].copy_(s["book0"])
    if own:
        zha = _lib()
        zha.pages_free(s["cfg"], s["pool"], s["dst"], ws=s["ws"])
        zha.pages_fork(s["cfg"], s["pool"], s["src"], s["dst"], s["fork_n"], ws=s["ws"])
        zha.pages_extend(s["cfg"], s["pool"], s["all"], s["new_n"], ws=s["ws"])
        return table, refs, s["K"], s["V"]
    src, dst, n = s["src"].long(), s["dst"].long(), s["fork_n"]
    block = torch.arange(table.shape[2], device="cuda")
    # the old beams' pages
    old = table[dst].flatten().long()
    refs.scatter_add_(0, old.clamp(min=0), -(old >= 0).int())
    # full blocks shared, the part-filled last one copied
    full = (block[None] < (n // C)[:, None])[:, None]
    new = torch.where(full, table[src], -1)
    shared = new.flatten().long()
    refs.scatter_add_(0, shared.clamp(min=0), (shared >= 0).int())
    part = (n % C > 0)[:, None].expand(-1, c["kv"])
    page = _take(refs, part)
    tail = (block[None] == (n // C)[:, None])[:, None] & part[..., None]
    table[dst] = torch.where(tail, page[..., None].int(), new)
    refs.scatter_add_(0, page.flatten().clamp(min=0), part.flatten().int())
    i, g = torch.nonzero(part, as_tuple=True)
    to, frm = page[i, g], table[src[i], g, n[i] // C].long()
    rows = (torch.arange(C, device="cuda")[None] < (n[i] % C)[:, None])[..., None]
    for x in (s["K"], s["V"]):
        x[to] = torch.where(rows, x[frm], x[to])
    # every sequence longer
    need = (block[None] < ((s["new_n"] + C - 1) // C)[:, None])[:, None] & (table < 0)
    page = _take(refs, need)
    table.copy_(torch.where(need, page.int(), table))
    refs.scatter_add_(0, page.flatten().clamp(min=0), need.flatten().int())
    return table, refs, s["K"], s["V"]


def _compact(s):
    table, refs = s["table"], s["refs"]
    s["book"].copy_(s["book0"])
    if own:
        _lib().pages_compact(s["cfg"], s["pool"], page_map=s["map"], n_live=s["live"], ws=s["ws"])
        return table, refs, s["map"], s["live"], s["K"], s["V"]
    live = refs > 0
    count = live.sum()
    at = torch.arange(refs.numel(), device="cuda")
    frm = torch.nonzero(live & (at >= count)).flatten()
    to = torch.nonzero(~live & (at < count)).flatten()
    for x in (s["K"], s["V"]):
        x[to] = x[frm]
    new = torch.where(live, at, -1)
    new[frm] = to
    refs[to] = refs[frm]
    refs[frm] = 0
    table.copy_(torch.where(table >= 0, new[table.clamp(min=0).long()].int(), table))
    s["map"].copy_(new)
    s["live"].copy_(count)
    return table, refs, s["map"], s["live"], s["K"], s["V"]


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    d = c["d"]
    if c["op"] == "attend":
        rows = sum(_spread(c["seqs"], c["tokens"])) * c["kv"]
        q = c["seqs"] * c["kv"] * c["group"]
        by = rows * 2 * d * ELT[c["cache"]] + q * (2 * d * ELT[c["q"]] + 4) + (rows / c["chunk"] * 4 if c["paged"] else 0) + 8 * c["seqs"]
        return {"bytes": by, "flops": rows * c["group"] * 4 * d}
    if c["op"] == "append":
        T, H, hq = c["new"], c["kv"], c["kv"] * c["group"]
        by = T * d * ((hq + 2 * H) * ELT[c["src"]] + hq * ELT[c["q"]] + 2 * H * ELT[c["cache"]]) + 20 * T + (4 * T * H / min(T, c["chunk"]) if c["paged"] else 0)
        return {"bytes": by, "flops": T * (hq + H) * c["pairs"] * 6}
    if c["op"] == "apply":
        T = c["new"]
        return {"bytes": T * c["heads"] * d * (ELT[c["src"]] + ELT[c["out"]]) + 8 * T, "flops": T * c["heads"] * c["pairs"] * 6}
    blocks, pages = _pages_layout(c)
    cells = c["slots"] * c["kv"] * blocks
    row = 2 * d * ELT[c["cache"]]
    book = 8 * (cells + pages)          # each pass starts from a copy of the table and counts
    if c["op"] == "beam":
        copied = c["forks"] * c["kv"] * (c["chunk"] - 1) / 2
        return {"bytes": book + 2 * copied * row + 4 * cells + 4 * pages, "flops": 0}
    live = 0.45 * min(1.0, c["live"] + 0.3) * min(1.0, 2 * c["live"])
    moved = pages * live * (1 - live) * c["chunk"]
    return {"bytes": book + 2 * moved * row + 8 * cells + 12 * pages, "flops": 0}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "attend":
        return _exact_attend(c, s)
    if c["op"] in ("append", "apply"):
        return _exact_rope(c, s)
    return _exact_pages(c, s)


def _exact_attend(c, s):
    S, H, G, d, C = c["seqs"], c["kv"], c["group"], c["d"], c["chunk"]
    o = torch.zeros(S, H * G, d, dtype=torch.float64, device="cuda")
    lse = torch.full((S, H * G), -math.inf, dtype=torch.float64, device="cuda")
    for i, n in enumerate(s["n"].tolist()):
        for h in range(H if n else 0):
            if s["table"] is None:
                k, v = s["K"][i, h, :n], s["V"][i, h, :n]
            else:
                pages = s["table"][i, h, : -(-n // C)].long()
                k, v = (x.index_select(0, pages).reshape(-1, d)[:n] for x in (s["K"], s["V"]))
            mine = slice(h * G, (h + 1) * G)
            w = (k.double() @ s["Q"][i, mine].double().T).T * d ** -0.5
            lse[i, mine] = torch.logsumexp(w, 1)
            o[i, mine] = torch.exp(w - lse[i, mine][:, None]) @ v.double()
    return o, lse


def _exact_thetas(c):
    a = _rope_args(c)
    D, base, f, out = 2 * c["pairs"], a["base"], a.get("factor", 1.0), []
    for i in range(c["pairs"]):
        t = base ** (-2.0 * i / D)
        if c["scaling"] == "linear":
            t /= f
        elif c["scaling"] == "ntk":
            t = (base * f ** (D / (D - 2))) ** (-2.0 * i / D) if D > 2 else t / f
        elif c["scaling"] == "yarn":
            edge = [D * math.log(a["original_tokens"] / (2 * math.pi * n)) / (2 * math.log(base)) for n in (a["high"], a["low"])]
            lo, hi = max(0, math.floor(edge[0])), min(c["pairs"] - 1, math.ceil(edge[1]))
            w = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            t = t * (1 - w) + t / f * w
        elif c["scaling"] == "bands":
            wave, L = 2 * math.pi / t, a["original_tokens"]
            if wave > L / a["low"]:
                t /= f
            elif wave >= L / a["high"]:
                w = (L / wave - a["low"]) / (a["high"] - a["low"])
                t = (1 - w) * t / f + w * t
        out.append(t)
    return np.array(out), 0.1 * math.log(f) + 1 if c["scaling"] == "yarn" else 1.0


def _exact_rope(c, s):
    theta, amp = _exact_thetas(c)
    P = c["pairs"]

    def turned(x, pos, sign):
        x = x.double().cpu().numpy()
        z = np.exp(1j * sign * pos.cpu().numpy()[:, None] * theta)[:, None] * amp
        first, second = (slice(0, P), slice(P, 2 * P)) if c["layout"] == "half" else (slice(0, 2 * P, 2), slice(1, 2 * P, 2))
        z = z * (x[..., first] + 1j * x[..., second])
        y = x.copy()
        y[..., first], y[..., second] = z.real, z.imag
        return torch.from_numpy(y)

    if c["op"] == "apply":
        return turned(s["X"], s["pos"], -1.0 if c["inverse"] else 1.0)
    H, C = c["kv"], c["chunk"]
    hq = H * c["group"]
    qkv = s["qkv"]
    k, v = turned(qkv[:, hq:hq + H], s["pos"], 1.0), qkv[:, hq + H:].double().cpu()
    K, V = (torch.zeros(x.shape, dtype=torch.float64) for x in (s["K"], s["V"]))
    seq, index = s["seq"].long().cpu(), s["index"].cpu()
    for h in range(H):
        for pool, x in ((K, k), (V, v)):
            if s["table"] is None:
                pool[seq, h, index] = x[:, h]
            else:
                pool[s["table"].cpu().long()[seq, h, index // C], index % C] = x[:, h]
    return turned(qkv[:, :hq], s["pos"], 1.0), K, V


def _exact_pages(c, s):
    C, K, V = c["chunk"], s["K"], s["V"]
    table, refs = s["table"].cpu().numpy().copy(), s["refs"].cpu().numpy().copy()
    S, H, B = table.shape
    if c["op"] == "compact":
        count = int((refs > 0).sum())
        holes = [p for p in range(count) if refs[p] == 0]
        name = [p if refs[p] > 0 else -1 for p in range(len(refs))]
        moved = [p for p in range(count, len(refs)) if refs[p] > 0]
        for p, to in zip(moved, holes):
            name[p], refs[to], refs[p] = to, refs[p], 0
        for x in (K, V):
            x[torch.tensor(holes, dtype=torch.long, device="cuda")] = x[torch.tensor(moved, dtype=torch.long, device="cuda")].clone()
        flat = table.reshape(-1)
        for j in range(flat.size):
            flat[j] = name[flat[j]] if flat[j] >= 0 else flat[j]
        return torch.from_numpy(table), torch.from_numpy(refs), torch.tensor(name, dtype=torch.int32), torch.tensor([count], dtype=torch.int32), K, V
    src, dst, n, new_n = (s[k].tolist() for k in ("src", "dst", "fork_n", "new_n"))
    for i in dst:
        for p in table[i].reshape(-1):
            if p >= 0:
                refs[p] -= 1
        table[i] = -1
    copies, free = [], [p for p in range(len(refs) - 1, -1, -1) if refs[p] == 0]
    for a, b, m in zip(src, dst, n):
        for h in range(H):
            table[b, h, : m // C] = table[a, h, : m // C]
            for p in table[b, h, : m // C]:
                refs[p] += 1
            if m % C:
                p = free.pop()
                refs[p] = 1
                table[b, h, m // C] = p
                copies.append((int(table[a, h, m // C]), p, m % C))
    for frm, to, rows in copies:
        K[to, :rows], V[to, :rows] = K[frm, :rows], V[frm, :rows]
    for i, m in enumerate(new_n):
        for h in range(H):
            for b in range(-(-m // C)):
                if table[i, h, b] < 0:
                    p = free.pop()
                    refs[p], table[i, h, b] = 1, p
    return torch.from_numpy(table), torch.from_numpy(refs), K, V
