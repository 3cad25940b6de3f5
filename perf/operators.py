"""Measured cases of the operators over the compressed KV cache that serve
speculative decoding and cache eviction:

  tree    attention of a tree of drafted tokens over the cache and the drafts
  commit  the accepted path of the tree stored behind the sequence
  mass    attention weight accumulated per cache position
  evict   the positions of largest weight copied into a smaller cache

``run`` computes them in plain torch (``own`` false) or through the
framework's entry points (``own`` true), on the same inputs: a cache buffer
in the layout of ``include/kvq.h`` and the tensors a decode loop has in hand.
``exact`` restates them in 64 bits from the quantised values themselves,
without reading the packed buffer."""
import math

import numpy as np
import torch

own = False

D = 128
SCALE = 1.0 / math.sqrt(D)
DEV = "cuda"

# Shapes of the repository's workloads: heads, visual range, bits, group size,
# protected heads (bf16 K and V).
TINY = dict(B=1, H_q=4, H_kv=1, vs=14, ve=256, kb=4, vb=4, G=32, prot="", konly="")
LLAVA_OV = dict(B=1, H_q=28, H_kv=4, vs=14, ve=6287, kb=4, vb=2, G=64, prot="0", konly="")
LLAVA15 = dict(B=16, H_q=32, H_kv=32, vs=40, ve=616, kb=8, vb=4, G=32, prot="3,11,20,29", konly="")
LLAVA_NEXT = dict(B=32, H_q=40, H_kv=40, vs=60, ve=2940, kb=4, vb=2, G=64, prot="1,9,17,25,33", konly="")


def _longctx(T):
    return dict(B=8, H_q=32, H_kv=8, vs=32, ve=T, kb=2, vb=2, G=32, prot="5", konly="")


def listed():
    return [
        # the smallest step: latency
        dict(TINY, name="tree_tiny_5", op="tree", T=257, T_cap=272, n_q=5, ragged=False, static=True),
        # one video sequence, 16 drafts (28/4 heads: 112 columns per KV head)
        dict(LLAVA_OV, name="tree_llava_ov_16", op="tree", T=6300, T_cap=6400, n_q=16, ragged=False, static=True),
        # a batch of image chats of unequal lengths, odd tree, one tree per sequence
        dict(LLAVA15, name="tree_llava15_ragged_26", op="tree", T=729, T_cap=760, n_q=26, ragged=True, static=False),
        # long context in 2 bits, a batch of 8
        dict(_longctx(16384), name="tree_longctx_16k_16", op="tree", T=16480, T_cap=16512, n_q=16, ragged=False, static=False),
        # the accepted path of one sequence
        dict(LLAVA_OV, name="commit_llava_ov", op="commit", T=6300, T_cap=6400, n_q=16, n_path=6, ragged=False),
        # ... of a batch, of unequal lengths
        dict(LLAVA15, name="commit_llava15_ragged", op="commit", T=729, T_cap=760, n_q=26, n_path=9, ragged=True),
        # after every decode step
        dict(LLAVA_OV, name="mass_llava_ov_1", op="mass", T=6288, T_cap=6400, n_q=1, ragged=False, path=False),
        dict(_longctx(32768), name="mass_longctx_32k_1", op="mass", T=32769, T_cap=32832, n_q=1, ragged=False, path=False),
        # an observation window of the prompt's last 32 tokens
        dict(LLAVA_NEXT, name="mass_llava_next_32", op="mass", T=2972, T_cap=3040, n_q=32, ragged=False, path=False),
        # half of a video's positions kept
        dict(LLAVA_OV, name="evict_llava_ov_half", op="evict", T=6487, T_cap=6600, keep_vis=3136, keep_text=100, recent=32, ragged=False),
        # a quarter of a long context, a batch of 8
        dict(_longctx(32768), name="evict_longctx_32k_8k", op="evict", T=32831, T_cap=32896, keep_vis=8160, keep_text=48, recent=16, ragged=False),
        # image chats of unequal lengths
        dict(LLAVA15, name="evict_llava15_ragged", op="evict", T=737, T_cap=760, keep_vis=144, keep_text=64, recent=17, ragged=True),
    ]


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "commit", "mass", "mass", "evict", "evict"])
    H_kv = rng.choice([1, 2, 3, 4, 5, 8, 16, 32])
    g = rng.choice([1, 1, 2, 3, 4, 5, 7, 8])
    B = rng.choice([1, 1, 2, 3, 5, 8, 16])
    n_vis = int(math.exp(rng.uniform(math.log(16), math.log(30000))))
    while B * H_kv * n_vis > 1000000:  # (sequence, head, position) triples: the largest listed case has twice as many
        n_vis //= 2
    vs = rng.randint(0, 70)
    n_suf = rng.randint(1, 200)
    heads = list(range(H_kv))
    rng.shuffle(heads)
    n_prot, n_konly = (rng.randint(0, 1 + H_kv // 8), rng.randint(0, 1)) if H_kv > 2 else (0, 0)
    T = vs + n_vis + n_suf
    c = dict(op=op, B=B, H_q=H_kv * g, H_kv=H_kv, vs=vs, ve=vs + n_vis, kb=rng.choice([2, 4, 4, 8, 16]),
             vb=rng.choice([2, 2, 4, 8, 16]), G=rng.choice([32, 64, 128]),
             prot=",".join(map(str, sorted(heads[:n_prot]))),
             konly=",".join(map(str, sorted(heads[n_prot:n_prot + n_konly]))), T=T, T_cap=T + rng.randint(64, 100),
             ragged=B > 1 and rng.random() < 0.5)
    if op == "tree":
        n_q = rng.randint(1, 64)
        while n_q > 1 and B * H_kv * g * n_q * n_vis > 60000000:  # (column, position) pairs
            n_q //= 2
        c.update(n_q=n_q, static=rng.random() < 0.5)
    elif op == "commit":
        n_q = rng.randint(1, 64)
        c.update(n_q=n_q, n_path=rng.randint(1, n_q))
    elif op == "mass":
        n_q = rng.choice([1, 1, 2, 3, 7, 16, 33, 64])
        while n_q > 1 and B * H_kv * g * n_q * n_vis > 60000000:
            n_q //= 2
        c.update(n_q=n_q, path=n_q > 1 and rng.random() < 0.5)
    else:
        keep_text = rng.randint(1, n_suf)
        c.update(keep_vis=int(n_vis * rng.uniform(0.05, 1.0)), keep_text=keep_text, recent=rng.randint(0, keep_text))
    return c


# ---- the cache buffer (the layout that include/kvq.h describes) ---------------

def _ints(text):
    return [int(x) for x in text.split(",") if x]


def _heads(c):
    """KV heads by kind: protected, K-only protected, packed."""
    prot, konly = _ints(c["prot"]), _ints(c["konly"])
    return prot, konly, [h for h in range(c["H_kv"]) if h not in prot and h not in konly]


def _segments(c):
    """(heads, rows per (sequence, head), bytes per row, offset) of the eight
    segments, and the buffer's size."""
    prot, konly, pack = _heads(c)
    Tv, B = c["ve"] - c["vs"], c["B"]
    Tvp, every = -(-Tv // 16) * 16, list(range(c["H_kv"]))
    sz = [0 if b == 16 else 4 * D // c["G"] for b in (c["kb"], c["vb"])]
    shapes = [(pack, Tvp, 16 * c["kb"]), (pack, Tvp, sz[0]), (pack + konly, Tvp, 16 * c["vb"]), (pack + konly, Tvp, sz[1]),
              (prot + konly, Tv, 2 * D), (prot, Tv, 2 * D), (every, c["T_cap"] - Tv, 2 * D), (every, c["T_cap"] - Tv, 2 * D)]
    spans = [-(-(B * len(h) * n * w + 256) // 256) * 256 for h, n, w in shapes]
    offs = [sum(spans[:i]) for i in range(9)]
    return [s + (o,) for s, o in zip(shapes, offs)], offs[8]


def _view(c, cache, i):
    """Segment i as uint8 [B, heads, rows, bytes]."""
    h, n, w, o = _segments(c)[0][i]
    return cache[o:o + c["B"] * len(h) * n * w].view(c["B"], len(h), n, w)


def _slots(bits, key):
    """Storage slot of each element d of a packed row."""
    if not key:
        return [16 * (d % 8) + 2 * (d // 16) + (d // 8) % 2 for d in range(D)]
    parts = [(d // 32, d % 32 // 8, d % 8 // 4, d % 4) for d in range(D)]
    if bits == 2:
        at = ((4, 7), (3, 6), (2, 5), (0, 1))
        return [32 * t + 16 * (i // 2) + 8 * e + at[P][i % 2] for P, t, e, i in parts]
    if bits == 4:
        return [32 * t + 8 * i + 4 * e + P for P, t, e, i in parts]
    return [32 * t + 4 * (2 * P + i // 2) + 2 * e + i % 2 for P, t, e, i in parts]


def _quantise(x, bits, G):
    """Codes, scales and zeros of bf16 rows [..., D]."""
    x = x.float().unflatten(-1, (D // G, G))
    lo = x.amin(-1) + 0.0
    s = ((x.amax(-1) - lo) / float(2 ** bits - 1)).half()
    z = lo.half()
    code = torch.round((x - z.float()[..., None]) / s.float()[..., None]).clamp(0, 2 ** bits - 1)
    code = torch.where(s[..., None] == 0, torch.zeros_like(code), code)
    return code.flatten(-2).to(torch.uint8), s, z


def _pack(code, bits, key):
    """uint8 codes [..., D] -> the stored bytes [..., D * bits / 8]."""
    place = torch.tensor(_slots(bits, key), device=code.device).argsort()
    per = 8 // bits
    shift = bits * torch.arange(per, device=code.device, dtype=torch.uint8)
    return (code[..., place].unflatten(-1, (-1, per)) << shift).sum(-1).to(torch.uint8)


def _bytes(x):
    return x.contiguous().view(torch.uint8)


def _fill(c, cache, key, x):
    """Store bf16 rows x [B, H_kv, >= T_cap, D] of K (key) or V."""
    prot, konly, pack = _heads(c)
    vs, ve, bits = c["vs"], c["ve"], c["kb"] if key else c["vb"]
    codes, szs, plain, text = (0, 1, 4, 6) if key else (2, 3, 5, 7)
    full, packed = (prot + konly, pack) if key else (prot, pack + konly)
    _view(c, cache, text)[:] = _bytes(torch.cat([x[:, :, :vs], x[:, :, ve:c["T_cap"]]], 2))
    if full and ve > vs:
        _view(c, cache, plain)[:] = _bytes(x[:, full, vs:ve])
    for i, h in enumerate(packed if ve > vs else []):
        rows = x[:, h, vs:ve]
        if bits == 16:
            _view(c, cache, codes)[:, i, :ve - vs] = _bytes(rows)
            continue
        code, s, z = _quantise(rows, bits, c["G"])
        _view(c, cache, codes)[:, i, :ve - vs] = _pack(code, bits, key)
        _view(c, cache, szs)[:, i, :ve - vs] = _bytes(torch.cat([z, s], -1))


def _places(c):
    """Byte of a packed row and shift inside it of each element, of K and V rows."""
    bit = [b * torch.tensor(_slots(b, key), device=DEV) for b, key in ((c["kb"], True), (c["vb"], False))]
    return [(b // 8, (b % 8).to(torch.uint8)) for b in bit]


def _read(c, cache, key, T, places):
    """Plain form: rows [0, T) of K (key) or V as fp32 [B, H_kv, T, D]."""
    prot, konly, pack = _heads(c)
    vs, ve, bits, n = c["vs"], min(c["ve"], T), c["kb"] if key else c["vb"], max(0, min(c["ve"], T) - c["vs"])
    codes, szs, plain, text = (0, 1, 4, 6) if key else (2, 3, 5, 7)
    full, packed = (prot + konly, pack) if key else (prot, pack + konly)
    tx = _view(c, cache, text).view(torch.bfloat16)
    if not n:
        return tx[:, :, :T].float()
    out = torch.empty(c["B"], c["H_kv"], T, D, device=cache.device)
    out[:, :, :vs] = tx[:, :, :vs].float()
    out[:, :, ve:] = tx[:, :, vs:vs + T - ve].float()
    if full:
        out[:, full, vs:ve] = _view(c, cache, plain).view(torch.bfloat16)[:, :, :n].float()
    if packed and bits == 16:
        out[:, packed, vs:ve] = _view(c, cache, codes).view(torch.bfloat16)[:, :, :n].float()
    elif packed:
        byte, shift = places[0] if key else places[1]
        code = (_view(c, cache, codes)[:, :, :n][..., byte] >> shift) & (2 ** bits - 1)
        zs = _view(c, cache, szs)[:, :, :n].view(torch.float16).float()
        z, s = zs.chunk(2, -1)
        out[:, packed, vs:ve] = (code.float().unflatten(-1, (-1, c["G"])) * s[..., None] + z[..., None]).flatten(-2)
    return out


# ---- inputs --------------------------------------------------------------------

def _lengths(c):
    """Lengths of the sequences: T, or unequal ones between the end of the
    visual block and T (the same for every seed, so that work() knows them)."""
    B, T, low = c["B"], c["T"], c["ve"]
    if not c["ragged"]:
        return [T] * B
    return [T - (T - low) * ((5 * b + 3) % B) // B for b in range(B)]


def _paths(c):
    """How many tokens of each sequence are taken (commit; mass with a path)."""
    n = c.get("n_path", c.get("n_q", 0))
    return [n - (3 * b) % (n + 1) for b in range(c["B"])]


def _rng(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _rows(c, r):
    """bf16 K and V rows [B, H_kv, T_cap, D]; K with a few channels of large
    magnitude per head, as rotated keys have."""
    shape = (c["B"], c["H_kv"], c["T_cap"], D)
    k = torch.randn(shape, device=DEV, dtype=torch.bfloat16, generator=r)
    loud = torch.ones(1, c["H_kv"], 1, D, device=DEV, dtype=torch.bfloat16)
    place = torch.rand(1, c["H_kv"], 1, D, device=DEV, generator=r).argsort(-1)[..., :4]
    k *= loud.scatter(-1, place, 8.0)
    return k, torch.randn(shape, device=DEV, dtype=torch.bfloat16, generator=r)


def _drafts(c, r):
    """K and V of the drafted tokens, as a projection leaves them
    ([B, n_q, H_kv, D]), seen as [B, H_kv, n_q, D]."""
    kv = torch.randn(2, c["B"], c["n_q"], c["H_kv"], D, device=DEV, dtype=torch.bfloat16, generator=r)
    return kv[0].transpose(1, 2), kv[1].transpose(1, 2)


def _tree(n_q, rows, seed):
    """Ancestor masks (bit j: token i sees draft j) of random trees, int64 [rows, n_q]."""
    g = np.random.default_rng(seed)
    masks = np.zeros((rows, n_q), np.uint64)
    for b in range(rows):
        for i in range(n_q):
            parent = int(g.integers(max(-1, i - 6), i)) if i else -1
            above = masks[b, parent] if parent >= 0 else np.uint64(0)
            masks[b, i] = above | np.uint64(1 << i)
    return masks.view(np.int64)


def _picked(c, seed):
    """Accepted tokens [B, n] in increasing order, int32 (entries behind
    a sequence's count are -1), and the counts."""
    g = np.random.default_rng(seed + 1)
    path, count = np.full((c["B"], c.get("n_path", c["n_q"])), -1, np.int32), np.array(_paths(c), np.int32)
    for b, n in enumerate(count):
        path[b, :n] = np.sort(g.permutation(c["n_q"])[:n])
    return path, count


def _smaller(c):
    """The case's eviction target as a cache of its own."""
    ve = c["vs"] + c["keep_vis"]
    return dict(c, ve=ve, T=ve + c["keep_text"], T_cap=ve + c["keep_text"] + 64)


def _sees(c, count, lens):
    """bool [B, n_q, T]: position t is attended by taken token k (causal at the end)."""
    k = torch.arange(c["n_q"], device=DEV)[None, :, None]
    t = torch.arange(c["T"], device=DEV)[None, None]
    return (k < count[:, None, None]) & (t < lens[:, None, None] - count[:, None, None] + 1 + k)


def _inputs(c, seed):
    """What the seed decides, without the cache buffer."""
    r = _rng(seed)
    s = {"k": None, "v": None}
    s["k"], s["v"] = _rows(c, r)
    s["lens"] = torch.tensor(_lengths(c), dtype=torch.int32, device=DEV)
    if c["op"] in ("tree", "commit"):
        s["kd"], s["vd"] = _drafts(c, r)
    if c["op"] in ("tree", "mass"):
        s["q"] = torch.randn(c["B"], c["n_q"], c["H_q"], D, device=DEV, dtype=torch.bfloat16, generator=r)
    if c["op"] == "tree":
        s["mask"] = torch.from_numpy(_tree(c["n_q"], 1 if c["static"] else c["B"], seed)).to(DEV)
    if c["op"] == "commit" or c.get("path"):
        s["path"], s["count"] = (torch.from_numpy(x).to(DEV) for x in _picked(c, seed))
    if c["op"] in ("mass", "evict"):
        w = torch.randn(c["B"], c["H_kv"], c["T_cap"], device=DEV, generator=r).mul_(2).exp_()
        # a weight that has underflowed, or a row nobody has looked at: exactly 0
        s["mass_in"] = w * (torch.rand(w.shape, device=DEV, generator=r) > 0.1)
    return s


def prepare(case, seed):
    c = case
    s = _inputs(c, seed)
    cache = torch.zeros(_segments(c)[1], dtype=torch.uint8, device=DEV)
    _fill(c, cache, True, s.pop("k"))
    _fill(c, cache, False, s.pop("v"))
    s.update(c=c, cache=cache, places=_places(c))
    B, n_q = c["B"], c.get("n_q", 0)
    if c["op"] == "tree":
        s["out"] = torch.zeros(B, n_q, c["H_q"], D, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.zeros(B, n_q, c["H_q"], device=DEV)
    elif c["op"] == "commit":
        s["new_len"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    elif c["op"] == "mass":
        # the lse that the attention of the same tokens returned
        count = s["count"] if c["path"] else torch.full((B,), n_q, dtype=torch.int32, device=DEV)
        q = _taken(c, s)
        score = SCALE * _columns(c, q.float()) @ _read(c, cache, True, c["T"], s["places"]).transpose(-1, -2)
        sees = _sees(c, count, s["lens"])[:, None, None]
        score = score.view(B, c["H_kv"], -1, n_q, c["T"]).masked_fill_(~sees, -math.inf)
        lse = torch.logsumexp(score, -1).permute(0, 3, 1, 2).reshape(B, n_q, c["H_q"]).contiguous()
        del score
        s["lse"] = lse
        if c["path"]:  # as the tree's tokens lie; the others' are finite and must not count
            s["lse"] = torch.full_like(lse, 3.0)
            b, i = (s["path"] >= 0).nonzero(as_tuple=True)
            s["lse"][b, s["path"].long()[b, i]] = lse[b, i]
        s["mass"] = torch.zeros_like(s["mass_in"])
    else:
        d = _smaller(c)
        s["dst"] = torch.zeros(_segments(d)[1], dtype=torch.uint8, device=DEV)
        s["keep"] = torch.zeros(B, c["H_kv"], d["T"], dtype=torch.int32, device=DEV)
        s["mass_dst"] = torch.zeros(B, c["H_kv"], d["T_cap"], device=DEV)
        s["new_len"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    if own:  # the handles and the workspace that a decode loop keeps
        s["L"] = _handle(c)
        if c["op"] == "tree":
            import bit_mixed_precision_kvq_gb300 as kvq
            s["ws"] = torch.zeros(kvq.decode_tree_workspace_bytes(s["L"], n_q), dtype=torch.uint8, device=DEV)
        if c["op"] == "evict":
            s["L_dst"] = _handle(_smaller(c))
    return s


def _handle(c):
    import bit_mixed_precision_kvq_gb300 as kvq
    L = kvq.cache_layout(c["B"], c["H_q"], c["H_kv"], D, c["T_cap"], c["vs"], c["ve"], c["kb"], c["vb"], c["G"],
                         _ints(c["prot"]), _ints(c["konly"]))
    assert int(L.total_bytes) == _segments(c)[1]
    return L


# ---- one pass --------------------------------------------------------------------

def run(state):
    c = state["c"]
    return (_run_own if own else _run_plain)[c["op"]](c, state)


def _own_tree(c, s):
    import bit_mixed_precision_kvq_gb300 as kvq
    kvq.decode_attention_tree(s["L"], s["cache"], s["q"], s["kd"], s["vd"], s["mask"], c["T"], s["out"], SCALE, s["lse"],
                              s["ws"], seq_len=s["lens"] if c["ragged"] else None)
    return s["out"], s["lse"]


def _own_commit(c, s):
    import bit_mixed_precision_kvq_gb300 as kvq
    kvq.tree_commit(s["L"], s["cache"], s["kd"], s["vd"], s["path"], s["count"], c["T"],
                    seq_len=s["lens"] if c["ragged"] else None, new_len=s["new_len"])
    return s["cache"], s["new_len"]


def _own_mass(c, s):
    import bit_mixed_precision_kvq_gb300 as kvq
    kvq.attention_mass(s["L"], s["cache"], s["q"], s["lse"], c["T"], s["mass"], s["mass_in"], SCALE, 0.98,
                       seq_len=s["lens"] if c["ragged"] else None, path=s.get("path"), path_len=s.get("count"))
    return s["mass"]


def _own_evict(c, s):
    import bit_mixed_precision_kvq_gb300 as kvq
    kvq.cache_evict(s["L"], s["cache"], s["mass_in"], c["T"], s["L_dst"], s["dst"], _smaller(c)["T"], s["keep"],
                    c["recent"], s["mass_dst"], seq_len=s["lens"] if c["ragged"] else None, new_len=s["new_len"])
    return s["dst"], s["keep"], s["mass_dst"], s["new_len"]


def _columns(c, q):
    """[B, n, H_q, D] -> [B, H_kv, g * n, D]."""
    B, n = q.shape[:2]
    return q.view(B, n, c["H_kv"], -1, D).permute(0, 2, 3, 1, 4).reshape(B, c["H_kv"], -1, D)


def _taken(c, s):
    """The queries in the order of the path (all of them without one)."""
    if not c["path"]:
        return s["q"]
    at = s["path"].clamp(min=0).long()[..., None, None].expand(-1, -1, c["H_q"], D)
    return s["q"].gather(1, at)


def _plain_tree(c, s):
    B, T, n_q, H = c["B"], c["T"], c["n_q"], c["H_kv"]
    k = torch.cat([_read(c, s["cache"], True, T, s["places"]), s["kd"].float()], 2)
    v = torch.cat([_read(c, s["cache"], False, T, s["places"]), s["vd"].float()], 2)
    score = SCALE * (_columns(c, s["q"].float()) @ k.transpose(-1, -2)).view(B, H, -1, n_q, T + n_q)
    past = (torch.arange(T, device=DEV) < s["lens"][:, None])[:, None].expand(B, n_q, T)
    tree = ((s["mask"][..., None] >> torch.arange(n_q, device=DEV)) & 1).bool().expand(B, n_q, n_q)
    sees = torch.cat([past, tree], 2)[:, None, None]
    score = torch.where(sees, score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, H, -1, T + n_q) @ v).view(B, H, -1, n_q, D) / torch.where(total == 0, torch.ones_like(total), total)
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(B, n_q, c["H_q"], D))
    s["lse"].copy_((top + torch.log(total))[..., 0].permute(0, 3, 1, 2).reshape(B, n_q, c["H_q"]))
    return s["out"], s["lse"]


def _plain_commit(c, s):
    n = s["path"].shape[1]
    ok = torch.arange(n, device=DEV)[None] < s["count"][:, None]
    b, i = ok.nonzero(as_tuple=True)
    row = s["lens"].long()[b] + i - (c["ve"] - c["vs"])
    text_k, text_v = (_view(c, s["cache"], x).view(torch.bfloat16) for x in (6, 7))
    j = s["path"].long()[b, i]
    text_k[b, :, row] = s["kd"][b, :, j]
    text_v[b, :, row] = s["vd"][b, :, j]
    s["new_len"].copy_(s["lens"] + s["count"])
    return s["cache"], s["new_len"]


def _plain_mass(c, s):
    B, T, n_q, H = c["B"], c["T"], c["n_q"], c["H_kv"]
    count = s["count"] if c["path"] else torch.full_like(s["lens"], n_q)
    lse = s["lse"]
    if c["path"]:
        lse = lse.gather(1, s["path"].clamp(min=0).long()[..., None].expand(-1, -1, c["H_q"]))
    score = SCALE * _columns(c, _taken(c, s).float()) @ _read(c, s["cache"], True, T, s["places"]).transpose(-1, -2)
    lse = lse.view(B, n_q, H, -1).permute(0, 2, 3, 1)[..., None]
    p = torch.exp(score.view(B, H, -1, n_q, T) - lse)
    p = torch.where(_sees(c, count, s["lens"])[:, None, None], p, torch.zeros_like(p)).sum((2, 3))
    live = (torch.arange(T, device=DEV) < s["lens"][:, None])[:, None]
    s["mass"][:, :, :T] = torch.where(live, 0.98 * s["mass_in"][:, :, :T] + p, s["mass"][:, :, :T])
    return s["mass"]


def _largest(w, live, n):
    """Positions of the n largest weights among the live ones, ties to the
    lowest, in increasing order; behind the last one, w.shape[-1]."""
    N = w.shape[-1]
    order = torch.where(live, w, torch.full_like(w, -math.inf)).sort(stable=True, dim=-1, descending=True)[1][..., :n]
    return torch.where(live.expand_as(w).gather(-1, order), order, torch.full_like(order, N)).sort(-1)[0]


def _chosen(c, w, lens):
    """Plain form of the selection: kept source positions [B, H_kv, T_dst], -1 behind the last."""
    d = _smaller(c)
    vs, ve, T = c["vs"], c["ve"], c["T"]
    B, H = w.shape[:2]
    vis = _largest(w[:, :, vs:ve], torch.ones(1, 1, ve - vs, dtype=torch.bool, device=DEV), c["keep_vis"]) + vs
    at = torch.arange(ve, T, device=DEV)[None, None]
    end = lens.view(B, 1, 1)
    text = torch.where(at >= end - c["recent"], torch.full((), math.inf, device=DEV), w[:, :, ve:T])
    text = _largest(text, (at < end).expand(B, H, T - ve), c["keep_text"]) + ve
    text = torch.where(text < T, text, torch.full_like(text, -1))
    pre = torch.arange(vs, device=DEV).expand(B, H, vs)
    assert d["T"] == vs + c["keep_vis"] + c["keep_text"]
    return torch.cat([pre, vis, text], 2)


def _move(c, d, src, dst, seg, at):
    """Rows `at` [B, H_kv, n] (-1: none) of a segment's heads to the front of the smaller cache's."""
    heads = _segments(c)[0][seg][0]
    if not heads or not at.shape[2]:
        return
    x, y, at = _view(c, src, seg), _view(d, dst, seg), at[:, heads]
    if not x.shape[3]:
        return
    rows = x.gather(2, at.clamp(min=0)[..., None].expand(-1, -1, -1, x.shape[3]))
    y[:, :, :at.shape[2]] = torch.where((at >= 0)[..., None], rows, y[:, :, :at.shape[2]])


def _plain_evict(c, s):
    d, vs, ve = _smaller(c), c["vs"], c["ve"]
    keep = _chosen(c, s["mass_in"], s["lens"])
    vis, text = keep[:, :, vs:d["ve"]] - vs, torch.cat([keep[:, :, :vs], keep[:, :, d["ve"]:]], 2)
    text = torch.where(text >= ve, text - (ve - vs), text)
    [_move(c, d, s["cache"], s["dst"], seg, vis if seg < 6 else text) for seg in range(8)]
    w = s["mass_in"].gather(2, keep.clamp(min=0))
    s["keep"].copy_(keep)
    s["mass_dst"].zero_()
    s["mass_dst"][:, :, :d["T"]] = torch.where(keep >= 0, w, torch.zeros_like(w))
    s["new_len"].copy_((keep[:, 0] >= 0).sum(-1))
    return s["dst"], s["keep"], s["mass_dst"], s["new_len"]


_run_own = {"tree": _own_tree, "commit": _own_commit, "mass": _own_mass, "evict": _own_evict}
_run_plain = {"tree": _plain_tree, "commit": _plain_commit, "mass": _plain_mass, "evict": _plain_evict}


# ---- what a pass cannot do without --------------------------------------------------

def _row_bytes(c, visual, key):
    """Bytes of the K (key) or V rows of one position, all KV heads."""
    prot, konly, pack = _heads(c)
    if not visual:
        return c["H_kv"] * 2 * D
    bits = c["kb"] if key else c["vb"]
    full, packed = (prot + konly, pack) if key else (prot, pack + konly)
    return len(full) * 2 * D + len(packed) * (16 * bits + (4 * D // c["G"] if bits < 16 else 0))


def work(case):
    c = case
    Tv, H, H_q, n_q = c["ve"] - c["vs"], c["H_kv"], c["H_q"], c.get("n_q", 0)
    lens = _lengths(c)
    rows = {key: sum(Tv * _row_bytes(c, True, key) + (n - Tv) * _row_bytes(c, False, key) for n in lens) for key in (True, False)}
    total = sum(lens)
    if c["op"] == "tree":
        small = c["B"] * n_q * (H_q * (4 * D + 4) + H * 4 * D) + 8 * n_q * (1 if c["static"] else c["B"])
        return {"bytes": rows[True] + rows[False] + small, "flops": 4 * D * H_q * n_q * (total + c["B"] * n_q // 2)}
    if c["op"] == "commit":
        n = sum(_paths(c))
        return {"bytes": 2 * n * H * 4 * D + 4 * n + 8 * c["B"], "flops": 0}
    if c["op"] == "mass":
        n = _paths(c) if c["path"] else [n_q] * c["B"]
        return {"bytes": rows[True] + 8 * H * total + sum(n) * H_q * (2 * D + 4), "flops": 2 * D * H_q * sum(a * b for a, b in zip(n, lens))}
    d = _smaller(c)
    kept = [min(n - c["ve"], c["keep_text"]) + c["vs"] for n in lens]
    moved = sum(c["keep_vis"] * _row_bytes(c, True, key) + k * _row_bytes(c, False, key) for k in kept for key in (True, False))
    return {"bytes": 4 * H * total + 2 * moved + 4 * c["B"] * H * (d["T"] + d["T_cap"]), "flops": 0}


# ---- the definition in 64 bits --------------------------------------------------------

def _values(c, x, key):
    """The values that the cache stands for, fp64 [B, H_kv, T_cap, D], from
    the bf16 rows x: visual rows of packed heads go through the quantiser."""
    prot, konly, pack = _heads(c)
    bits, out = c["kb"] if key else c["vb"], x.double()
    if bits < 16 and c["ve"] > c["vs"]:
        for h in pack if key else pack + konly:
            code, s, z = _quantise(x[:, h, c["vs"]:c["ve"]], bits, c["G"])
            g = torch.arange(D, device=DEV) // c["G"]
            out[:, h, c["vs"]:c["ve"]] = code.double() * s.double()[..., g] + z.double()[..., g]
    return out


def exact(case, seed):
    c = case
    s = _inputs(c, seed)
    if c["op"] == "commit":
        return None  # rows are copied: nothing is computed
    lens = s["lens"].tolist()
    B, H, g, T = c["B"], c["H_kv"], c["H_q"] // c["H_kv"], c["T"]
    if c["op"] == "evict":
        return _exact_evict(c, s["mass_in"], lens)
    if c["op"] == "tree":
        K, V = _values(c, s["k"], True), _values(c, s["v"], False)
        out = torch.zeros(B, c["n_q"], c["H_q"], D, dtype=torch.float64, device=DEV)
        lse = torch.zeros(B, c["n_q"], c["H_q"], dtype=torch.float64, device=DEV)
        masks = s["mask"].expand(B, -1).cpu().tolist()
        for b in range(B):
            sees = torch.ones(c["n_q"], lens[b] + c["n_q"], dtype=torch.bool, device=DEV)
            sees[:, lens[b]:] = torch.tensor([[(m >> j) & 1 for j in range(c["n_q"])] for m in masks[b]], dtype=torch.bool)
            for h in range(H):
                k = torch.cat([K[b, h, :lens[b]], s["kd"][b, h].double()])
                v = torch.cat([V[b, h, :lens[b]], s["vd"][b, h].double()])
                for j in range(h * g, h * g + g):
                    a = (s["q"][b, :, j].double() @ k.T * SCALE).masked_fill(~sees, -math.inf)
                    out[b, :, j] = torch.softmax(a, -1) @ v
                    lse[b, :, j] = torch.logsumexp(a, -1)
        return out, lse
    state = prepare(dict(c), seed)
    given, K = state["lse"].double(), _values(c, s["k"], True)
    mass = torch.zeros(B, H, c["T_cap"], dtype=torch.float64, device=DEV)
    for b in range(B):
        path = s["path"][b, :s["count"][b]].tolist() if c["path"] else list(range(c["n_q"]))
        n = len(path)
        end = lens[b] - n + 1 + torch.arange(n, device=DEV)
        late = torch.arange(lens[b], device=DEV)[None] >= end[:, None]
        for h in range(H):
            q = s["q"][b, path, h * g:h * g + g].double()
            a = torch.einsum("njd,td->njt", q, K[b, h, :lens[b]]) * SCALE - given[b, path, h * g:h * g + g, None]
            mass[b, h, :lens[b]] = 0.98 * s["mass_in"][b, h, :lens[b]].double() + a.exp().masked_fill(late[:, None], 0.0).sum((0, 1))
    return mass


def _exact_evict(c, w, lens):
    d, vs, ve = _smaller(c), c["vs"], c["ve"]
    w = w.double().cpu().numpy()
    keep = np.full((c["B"], c["H_kv"], d["T"]), -1, np.int32)
    mass = np.zeros((c["B"], c["H_kv"], d["T_cap"]))
    for b in range(c["B"]):
        for h in range(c["H_kv"]):
            x = w[b, h]
            vis = vs + np.argsort(-x[vs:ve], kind="stable")[:c["keep_vis"]]
            old = max(ve, lens[b] - c["recent"])
            room = c["keep_text"] - (lens[b] - old)
            text = ve + np.argsort(-x[ve:old], kind="stable")[:room]
            at = np.concatenate([np.arange(vs), np.sort(vis), np.sort(text), np.arange(old, lens[b])])
            keep[b, h, :len(at)] = at
            mass[b, h, :len(at)] = x[at]
    return None, torch.from_numpy(keep).to(DEV), torch.from_numpy(mass).to(DEV), torch.from_numpy((keep[:, 0] >= 0).sum(-1).astype(np.int32))
