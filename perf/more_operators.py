"""Measured cases of the operators around a decode step over the compressed KV
cache:

  rope    norms of the query and key heads and their rotation by positions of
          several axes, from the projection's output to what the cache's calls take
  verify  drafted tokens held against the target's logits: the accepted path
          and the token behind it
  window  decode attention over the first positions and the last ones

``run`` computes them in plain torch (``own`` false) or through the
framework's entry points (``own`` true), on the same inputs. ``exact``
restates them in 64 bits."""
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
LONG = dict(B=8, H_q=32, H_kv=8, vs=32, ve=32768, kb=2, vb=2, G=32, prot="5", konly="")


def listed():
    return [
        # one token of one sequence before its decode step: latency
        dict(name="rope_step_llava_ov", op="rope", B=1, n=1, H_q=28, H_kv=4, R=128, axes="16,24,24", pair=False, norm=False),
        # drafted tokens of a batch, heads normed, interleaved pairs, part of the head rotated
        dict(name="rope_drafts_llava15", op="rope", B=16, n=26, H_q=32, H_kv=32, R=96, axes="48", pair=True, norm=True),
        # a batch of image prompts: time, height and width
        dict(name="rope_prompt_llava_next", op="rope", B=8, n=2940, H_q=40, H_kv=40, R=128, axes="16,24,24", pair=False, norm=True),
        # a few drafts of one sequence, the smallest vocabulary: latency
        dict(name="verify_5", op="verify", B=1, n_q=5, V=32000, half=True, probs=False, ragged=False, cold=0, heat=1.0, rows=1.8),
        # drafts sampled from a smaller model, its probabilities at hand, a large vocabulary
        dict(name="verify_probs_16", op="verify", B=1, n_q=16, V=152000, half=True, probs=True, ragged=False, cold=0, heat=0.8, rows=4.2),
        # a batch of unequal trees, a quarter of the sequences greedy, odd vocabulary, fp32 logits
        dict(name="verify_ragged_26", op="verify", B=16, n_q=26, V=32003, half=False, probs=False, ragged=True, cold=4, heat=1.0, rows=2.2),
        # a large batch with the largest trees
        dict(name="verify_probs_64", op="verify", B=32, n_q=64, V=128000, half=True, probs=True, ragged=False, cold=0, heat=1.0, rows=4.2),
        # the smallest step: latency
        dict(TINY, name="window_tiny", op="window", T=257, T_cap=272, n_q=1, n_sink=4, window=128, ragged=False),
        # one video sequence
        dict(LLAVA_OV, name="window_llava_ov_2k", op="window", T=6300, T_cap=6400, n_q=1, n_sink=30, window=2048, ragged=False),
        # four drafted tokens of image chats of unequal lengths
        dict(LLAVA15, name="window_llava15_ragged_4", op="window", T=729, T_cap=760, n_q=4, n_sink=44, window=301, ragged=True),
        # a long context in 2 bits, a quarter of it in the window
        dict(LONG, name="window_longctx_8k", op="window", T=32800, T_cap=32832, n_q=1, n_sink=64, window=8192, ragged=False),
        # sixteen drafted tokens of a large batch of image chats
        dict(LLAVA_NEXT, name="window_llava_next_16", op="window", T=2972, T_cap=3040, n_q=16, n_sink=64, window=1024, ragged=False),
    ]


def _log(rng, low, high):
    return int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))


def draw(rng):
    op = rng.choice(["rope", "verify", "window", "window"])
    if op == "rope":
        H_kv, g = rng.choice([1, 2, 3, 4, 5, 8, 16, 32]), rng.choice([1, 2, 3, 4, 5, 7, 8])
        B, n, R = _log(rng, 1, 32), _log(rng, 1, 8000), 8 * rng.randint(1, 16)
        while B * n * H_kv * (g + 1) > 1800000:  # rows: the largest listed case has 1.9 million
            n = n // 2 + 1 if n > 2 else 1
            B = B if n > 1 else B // 2
        cuts = sorted(rng.randint(0, R // 2) for _ in range(rng.randint(0, 3)))
        axes = ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [R // 2]))
        return dict(op=op, B=B, n=n, H_q=H_kv * g, H_kv=H_kv, R=R, axes=axes, pair=rng.random() < 0.4, norm=rng.random() < 0.5)
    if op == "verify":
        B, n_q, V = _log(rng, 1, 32), _log(rng, 1, 64), _log(rng, 500, 256000)
        while B * n_q * V > 262000000:  # logits: as many as the largest listed case has
            n_q = n_q // 2 + 1 if n_q > 2 else 1
            B = B if n_q > 1 else B // 2
        return dict(op=op, B=B, n_q=n_q, V=V, half=rng.random() < 0.5, probs=rng.random() < 0.5, ragged=rng.random() < 0.5,
                    cold=rng.choice([0, 0, 3]), heat=rng.choice([0.6, 0.9, 1.0, 1.3]), rows=min(4.0, 1.0 + 0.35 * n_q ** 0.5))
    H_kv, g = rng.choice([1, 2, 3, 4, 5, 8, 16, 32, 40]), rng.choice([1, 1, 2, 3, 4, 5, 7, 8])
    B, n_vis = rng.choice([1, 1, 2, 3, 5, 8, 16, 32]), _log(rng, 16, 30000)
    while B * H_kv * n_vis > 2000000:  # (sequence, head, position) triples of the cache: the largest listed case's
        n_vis //= 2
    vs, n_suf = rng.randint(0, 70), rng.randint(8, 200)
    heads = list(range(H_kv))
    rng.shuffle(heads)
    n_prot, n_konly = (rng.randint(0, 1 + H_kv // 8), rng.randint(0, 1)) if H_kv > 2 else (0, 0)
    T = vs + n_vis + n_suf
    n_q, n_sink, window = rng.choice([1, 1, 1, 2, 3, 4, 7, 8, 16, 33, 64]), rng.choice([0, 1, 4, 16, 33, 64, 128]), _log(rng, 1, T)
    n_q = min(n_q, n_suf)
    while B * H_kv * (n_sink + window + n_q) > 1400000:  # triples that are read, and (column, position) pairs: the largest listed case's
        window //= 2
    while B * H_kv * g * n_q * (n_sink + window + n_q) > 23000000:
        n_q //= 2
    return dict(op=op, B=B, H_q=H_kv * g, H_kv=H_kv, vs=vs, ve=vs + n_vis, kb=rng.choice([2, 4, 4, 8, 16]),
                vb=rng.choice([2, 2, 4, 8, 16]), G=rng.choice([32, 64, 128]),
                prot=",".join(map(str, sorted(heads[:n_prot]))), konly=",".join(map(str, sorted(heads[n_prot:n_prot + n_konly]))),
                T=T, T_cap=T + rng.randint(0, 60), n_q=n_q, n_sink=n_sink, window=window,
                ragged=B > 1 and rng.random() < 0.5)


def _rng(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _ints(text):
    return [int(x) for x in text.split(",") if x]


# ---- rope: norms and rotation ------------------------------------------------------

EPS = 1e-6


def _axis(c):
    """The position axis of each rotated pair."""
    return [a for a, n in enumerate(_ints(c["axes"])) for _ in range(n)]


def _pairs(c):
    """Elements (first, second) of each rotated pair."""
    i = torch.arange(c["R"] // 2, device=DEV)
    return (2 * i, 2 * i + 1) if c["pair"] else (i, i + c["R"] // 2)


def _rope_inputs(c, seed):
    r = _rng(seed)
    B, n, n_axes = c["B"], c["n"], len(_ints(c["axes"]))
    qkv = torch.randn(B, n, c["H_q"] + 2 * c["H_kv"], D, device=DEV, dtype=torch.bfloat16, generator=r)
    s = {"q": qkv[:, :, :c["H_q"]], "k": qkv[:, :, c["H_q"]:c["H_q"] + c["H_kv"]]}
    # frames of 14 x 14 patches behind a text of some length: time, height, width (and one more)
    start = torch.randint(0, 30000, (1, B, 1), device=DEV, dtype=torch.int32, generator=r)
    at = torch.arange(n, device=DEV, dtype=torch.int32)
    s["pos"] = (torch.stack([at // 196, at // 14 % 14, at % 14, at][:n_axes] if n_axes > 1 else [at])[:, None] + start).contiguous()
    s["freq"] = (1e6 ** (-torch.arange(c["R"] // 2, device=DEV, dtype=torch.float64) * 2 / c["R"])).float()
    for x in ("q", "k"):
        s[x + "_weight"] = (1 + 0.3 * torch.randn(D, device=DEV, generator=r)).bfloat16() if c["norm"] else None
    return s


def _prepare_rope(c, seed):
    s = _rope_inputs(c, seed)
    s.update(c=c, first=_pairs(c)[0], second=_pairs(c)[1], axis=torch.tensor(_axis(c), device=DEV))
    s["q_out"] = torch.zeros(c["B"], c["n"], c["H_q"], D, device=DEV, dtype=torch.bfloat16)
    # K as the cache's append and the tree's drafts take it
    s["k_out"] = torch.zeros(c["B"], c["H_kv"], c["n"], D, device=DEV, dtype=torch.bfloat16)
    if own:
        import bit_mixed_precision_kvq_gb300 as kvq
        s["L"] = kvq.cache_layout(c["B"], c["H_q"], c["H_kv"], D, c["n"], 0, 0, 4, 4, 32)
        s["R"] = kvq.rope_desc(c["R"], _axis(c), interleaved=c["pair"])
    return s


def _own_rope(c, s):
    import bit_mixed_precision_kvq_gb300 as kvq
    kvq.norm_rope(s["L"], s["R"], s["q"], s["k"], s["pos"], s["freq"], s["q_out"], s["k_out"].transpose(1, 2),
                  q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS)
    return s["q_out"], s["k_out"]


def _plain_rope(c, s):
    # angles in 64 bits: positions are large
    angle = (s["pos"][s["axis"]].double() * s["freq"].double()[:, None, None]).permute(1, 2, 0)[:, :, None]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    for x, out in (("q", s["q_out"]), ("k", s["k_out"].transpose(1, 2))):
        y = s[x].float()
        if c["norm"]:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * s[x + "_weight"].float()
        a, b = y[..., s["first"]], y[..., s["second"]]
        out.copy_(y)
        out[..., s["first"]] = (a * cos - b * sin).bfloat16()
        out[..., s["second"]] = (b * cos + a * sin).bfloat16()
    return s["q_out"], s["k_out"]


def _exact_rope(c, seed):
    s, R = _rope_inputs(c, seed), c["R"]
    freq, axis = s["freq"].double(), torch.tensor(_axis(c), device=DEV)
    turn = torch.polar(torch.ones((), device=DEV, dtype=torch.float64), s["pos"][axis].permute(1, 2, 0).double() * freq)
    res = []
    for x in ("q", "k"):
        out = []
        for b in range(c["B"]):  # one sequence at a time: 64 bits take room
            y = s[x][b].double()
            if c["norm"]:
                y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + EPS) * s[x + "_weight"].double()
            z = torch.complex(y[..., 0:R:2], y[..., 1:R:2]) if c["pair"] else torch.complex(y[..., :R // 2], y[..., R // 2:R])
            z = z * turn[b][:, None]
            w = torch.view_as_real(z).flatten(-2) if c["pair"] else torch.cat([z.real, z.imag], -1)
            out.append(torch.cat([w, y[..., R:]], -1).float())  # kept in 32 bits: the outputs have 8
        res.append(torch.stack(out))
    return res[0], res[1].transpose(1, 2).contiguous()


# ---- verify: drafted tokens and the target's logits ----------------------------------

def _sizes(c):
    """Tokens of each sequence's tree."""
    return [c["n_q"] if not c["ragged"] else 1 + (c["n_q"] - 1) * ((5 * b + 3) % (c["B"] + 1)) // max(1, c["B"]) for b in range(c["B"])]


def _trees(c, seed):
    """Parents and ancestor masks (bit j: token i follows j, its own bit set) of
    random trees below token 0, and how many earlier siblings each token has."""
    g = np.random.default_rng(seed)
    B, n = c["B"], c["n_q"]
    parent, mask, rank = np.full((B, n), -1), np.ones((B, n), np.uint64), np.zeros((B, n), np.int64)
    for j in range(1, n):
        parent[:, j] = g.integers(max(0, j - 6), j, B)
        mask[:, j] = mask[np.arange(B), parent[:, j]] | np.uint64(1 << j)
        rank[:, j] = (parent[:, :j] == parent[:, j:j + 1]).sum(1)
    return parent, mask, rank


def _verify_inputs(c, seed):
    r = _rng(seed)
    B, n, V = c["B"], c["n_q"], c["V"]
    parent, mask, rank = _trees(c, seed)
    # a likely token per row, of probability 0.1 to 0.95, over a broad rest
    x = torch.randn(B, n, V, device=DEV, generator=r).mul_(2.5)
    best = torch.randint(0, V, (B, n, 1), device=DEV, generator=r)
    x.scatter_(2, best, (math.log(V) + 3.1 + 1.5 * torch.randn(B, n, 1, device=DEV, generator=r)))
    logits = x.bfloat16() if c["half"] else x
    # the draft model: the same with noise
    x = x + 0.4 * torch.randn(B, n, V, device=DEV, generator=r)
    up, at = torch.from_numpy(parent).clamp(min=0).to(DEV), torch.from_numpy(rank).to(DEV)
    width = int(rank.max()) + 1
    if c["probs"]:  # siblings are drawn one by one from their parent's distribution
        draft = torch.softmax(x, -1)
        kids = torch.multinomial(draft.view(-1, V), width, replacement=True, generator=r).view(B, n, width)
    else:  # siblings are the most likely ones
        draft = None
        kids = x.topk(width, -1).indices
    del x
    tokens = kids.gather(1, up[..., None].expand(-1, -1, width)).gather(2, at[..., None])[..., 0].int()
    heat = [0.0 if c["cold"] and b % c["cold"] == c["cold"] - 1 else c["heat"] for b in range(B)]
    return dict(logits=logits, draft=draft, tokens=tokens, mask=torch.from_numpy(mask.view(np.int64)).to(DEV),
                heat=torch.tensor(heat, device=DEV), size=torch.tensor(_sizes(c), dtype=torch.int32, device=DEV),
                accept=torch.rand(B, n, device=DEV, generator=r), race=torch.empty(B, V, device=DEV).exponential_(generator=r),
                parent=parent)


def _prepare_verify(c, seed):
    s = _verify_inputs(c, seed)
    B, n = c["B"], c["n_q"]
    s.update(c=c, path=torch.zeros(B, n, dtype=torch.int32, device=DEV), count=torch.zeros(B, dtype=torch.int32, device=DEV),
             token=torch.zeros(B, dtype=torch.int32, device=DEV), logp=torch.zeros(B, n, device=DEV))
    return s


def _own_verify(c, s):
    import bit_mixed_precision_kvq_gb300 as kvq
    kvq.tree_verify(s["logits"], s["tokens"], s["mask"], s["accept"], s["race"], s["path"], s["count"], s["token"],
                    draft_prob=s["draft"], temperature=s["heat"], tree_len=s["size"], logprob=s["logp"])
    return s["path"], s["count"], s["token"], s["logp"]


def _first_best(x):
    """Lowest index of each row's largest value."""
    at = torch.arange(x.shape[-1], device=DEV).expand_as(x)
    return torch.where(x == x.amax(-1, keepdim=True), at, torch.full_like(at, x.shape[-1])).amin(-1)


def _plain_verify(c, s):
    # probabilities in 64 bits: a random number may lie next to the border
    B, n, V = c["B"], c["n_q"], c["V"]
    each, at = torch.arange(B, device=DEV), torch.arange(n, device=DEV)
    below = ((s["mask"][..., None] >> at) & 1).bool() & (at < at[:, None])
    parent = torch.where(below, at, torch.full_like(at, -1)).amax(-1)
    greedy = s["heat"] <= 0
    inv = 1 / torch.where(greedy, torch.ones_like(s["heat"]), s["heat"]).double()

    def row(cur):
        x = s["logits"][each, cur].double() * inv[:, None]
        top = x.amax(-1, keepdim=True)
        lse = top + torch.log(torch.exp(x - top).sum(-1, keepdim=True))
        return x - lse, torch.exp(x - lse), _first_best(x)

    cur, count = torch.zeros_like(each), torch.ones_like(each)
    logp_row, rest, best = row(cur)
    total = torch.ones(B, device=DEV, dtype=torch.float64)
    s["path"].fill_(-1)
    s["path"][:, 0] = 0
    s["logp"].zero_()
    for j in range(1, n):  # a token's parent and earlier siblings lie before it
        token = s["tokens"][:, j].long()[:, None]
        tried = (parent[:, j] == cur) & (j < s["size"])
        won = torch.where(greedy, token[:, 0] == best, s["accept"][:, j].double() * total * (s["draft"][each, cur].gather(1, token)[:, 0].double() if c["probs"] else 1.0)
                          < rest.gather(1, token)[:, 0])
        took, lost = tried & won, tried & ~won
        s["logp"][each, count - 1] = torch.where(took, logp_row.gather(1, token)[:, 0].float(), s["logp"][each, count - 1])
        if c["probs"]:
            left = (rest / total[:, None] - s["draft"][each, cur].double()).clamp_(min=0)
        else:
            left = rest.scatter(1, token, 0.0)
        rest = torch.where(lost[:, None], left, rest)
        total = torch.where(lost, rest.sum(-1), total)
        cur, count = torch.where(took, j, cur), count + took
        s["path"][each, count - 1] = cur.int()
        logp_row, fresh, best = row(cur)
        rest = torch.where(took[:, None], fresh, rest)
        total = torch.where(took, torch.ones_like(total), total)
    key = rest / s["race"].double()
    token = torch.where(greedy | (key.amax(-1) == 0), best, _first_best(key))
    s["logp"][each, count - 1] = logp_row.gather(1, token[:, None])[:, 0].float()
    s["count"].copy_(count)
    s["token"].copy_(token)
    return s["path"], s["count"], s["token"], s["logp"]


def _exact_verify(c, seed):
    s = _verify_inputs(c, seed)
    B, n = c["B"], c["n_q"]
    parent, sizes, heat = s["parent"], _sizes(c), s["heat"].double().cpu().numpy()
    u, tokens = s["accept"].double().cpu().numpy(), s["tokens"].cpu().numpy()
    path, count, token, logp = np.full((B, n), -1, np.int32), np.zeros(B, np.int32), np.zeros(B, np.int32), np.zeros((B, n))
    for b in range(B):
        walk, cur = [0], 0
        while True:
            x = s["logits"][b, cur].double().cpu().numpy() / (heat[b] if heat[b] > 0 else 1.0)
            x -= x.max()
            lp = x - np.log(np.exp(x).sum())
            p, q = np.exp(lp), s["draft"][b, cur].double().cpu().numpy() if c["probs"] else None
            goes = None
            for j in [j for j in range(1, sizes[b]) if parent[b, j] == cur]:
                t = tokens[b, j]
                if heat[b] <= 0:
                    ok = t == int(np.argmax(lp))
                elif c["probs"]:
                    ok = u[b, j] * q[t] < p[t]
                    p = p if ok else np.maximum(p - q, 0) / np.maximum(p - q, 0).sum()
                else:
                    ok = u[b, j] < p[t]
                    if not ok:
                        p[t] = 0
                        p /= p.sum()
                if ok:
                    goes = j
                    break
            if goes is None:
                break
            logp[b, len(walk) - 1] = lp[tokens[b, goes]]
            walk.append(goes)
            cur = goes
        token[b] = int(np.argmax(lp)) if heat[b] <= 0 else int(np.argmax(p / s["race"][b].double().cpu().numpy()))
        logp[b, len(walk) - 1] = lp[token[b]]
        path[b, :len(walk)], count[b] = walk, len(walk)
    return tuple(torch.from_numpy(x) for x in (path, count, token, logp))


# ---- window: the cache buffer (the layout that include/kvq.h describes) ----------------

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
    """Store bf16 rows x [B, H_kv, T_cap, D] of K (key) or V."""
    prot, konly, pack = _heads(c)
    vs, ve, bits = c["vs"], c["ve"], c["kb"] if key else c["vb"]
    codes, szs, plain, text = (0, 1, 4, 6) if key else (2, 3, 5, 7)
    full, packed = (prot + konly, pack) if key else (prot, pack + konly)
    _view(c, cache, text)[:] = _bytes(torch.cat([x[:, :, :vs], x[:, :, ve:]], 2))
    if full:
        _view(c, cache, plain)[:] = _bytes(x[:, full, vs:ve])
    for i, h in enumerate(packed):
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


def _read(c, cache, key, lo, hi, places):
    """Plain form: rows [lo, hi) of K (key) or V as fp32 [B, H_kv, hi - lo, D]."""
    prot, konly, pack = _heads(c)
    vs, ve, bits = c["vs"], c["ve"], c["kb"] if key else c["vb"]
    codes, szs, plain, text = (0, 1, 4, 6) if key else (2, 3, 5, 7)
    full, packed = (prot + konly, pack) if key else (prot, pack + konly)
    tx = _view(c, cache, text).view(torch.bfloat16)
    out = torch.empty(c["B"], c["H_kv"], hi - lo, D, device=cache.device)
    pre, a, b = min(vs, hi), max(vs, lo), max(vs, min(ve, hi))  # visual part [a, b)
    a = min(a, b)
    if lo < pre:
        out[:, :, :pre - lo] = tx[:, :, lo:pre].float()
    if hi > max(ve, lo):
        out[:, :, max(ve, lo) - lo:] = tx[:, :, max(ve, lo) - (ve - vs):hi - (ve - vs)].float()
    if a < b:
        if full:
            out[:, full, a - lo:b - lo] = _view(c, cache, plain).view(torch.bfloat16)[:, :, a - vs:b - vs].float()
        if packed and bits == 16:
            out[:, packed, a - lo:b - lo] = _view(c, cache, codes).view(torch.bfloat16)[:, :, a - vs:b - vs].float()
        elif packed:
            byte, shift = places[0] if key else places[1]
            code = (_view(c, cache, codes)[:, :, a - vs:b - vs][..., byte] >> shift) & (2 ** bits - 1)
            zs = _view(c, cache, szs)[:, :, a - vs:b - vs].view(torch.float16).float()
            z, s = zs.chunk(2, -1)
            out[:, packed, a - lo:b - lo] = (code.float().unflatten(-1, (-1, c["G"])) * s[..., None] + z[..., None]).flatten(-2)
    return out


def _lengths(c):
    """Lengths of the sequences: T, or unequal ones between the end of the
    visual block (and the tokens' own rows) and T, the same for every seed."""
    B, T, low = c["B"], c["T"], c["ve"] + c["n_q"]
    if not c["ragged"]:
        return [T] * B
    return [T - (T - low) * ((5 * b + 3) % B) // B for b in range(B)]


def _window_inputs(c, seed):
    r = _rng(seed)
    shape = (c["B"], c["H_kv"], c["T_cap"], D)
    k = torch.randn(shape, device=DEV, dtype=torch.bfloat16, generator=r)
    # a few channels of large magnitude per head, as rotated keys have
    loud = torch.ones(1, c["H_kv"], 1, D, device=DEV, dtype=torch.bfloat16)
    place = torch.rand(1, c["H_kv"], 1, D, device=DEV, generator=r).argsort(-1)[..., :4]
    k *= loud.scatter(-1, place, 8.0)
    v = torch.randn(shape, device=DEV, dtype=torch.bfloat16, generator=r)
    q = torch.randn(c["B"], c["n_q"], c["H_q"], D, device=DEV, dtype=torch.bfloat16, generator=r)
    return k, v, q, torch.tensor(_lengths(c), dtype=torch.int32, device=DEV)


def _prepare_window(c, seed):
    k, v, q, lens = _window_inputs(c, seed)
    cache = torch.zeros(_segments(c)[1], dtype=torch.uint8, device=DEV)
    _fill(c, cache, True, k)
    _fill(c, cache, False, v)
    s = dict(c=c, cache=cache, q=q, lens=lens, places=_places(c), out=torch.zeros_like(q),
             lse=torch.zeros(q.shape[:3], device=DEV))
    if own:
        import bit_mixed_precision_kvq_gb300 as kvq
        s["L"] = kvq.cache_layout(c["B"], c["H_q"], c["H_kv"], D, c["T_cap"], c["vs"], c["ve"], c["kb"], c["vb"], c["G"],
                                  _ints(c["prot"]), _ints(c["konly"]))
        assert int(s["L"].total_bytes) == _segments(c)[1]
    return s


def _own_window(c, s):
    import bit_mixed_precision_kvq_gb300 as kvq
    kvq.decode_attention_window(s["L"], s["cache"], s["q"], c["T"], c["n_sink"], c["window"], s["out"], SCALE, s["lse"],
                                seq_len=s["lens"] if c["ragged"] else None)
    return s["out"], s["lse"]


def _plain_window(c, s):
    B, H, n = c["B"], c["H_kv"], c["n_q"]
    # positions that some token of some sequence may see: the first ones, and from the earliest window on
    lo = max(min(c["n_sink"], c["T"]), (min(_lengths(c)) if c["ragged"] else c["T"]) - n + 1 - c["window"])
    first = min(c["n_sink"], c["T"])
    k, v = (torch.cat([_read(c, s["cache"], key, 0, first, s["places"]), _read(c, s["cache"], key, lo, c["T"], s["places"])], 2) for key in (True, False))
    t = torch.cat([torch.arange(first, device=DEV), torch.arange(lo, c["T"], device=DEV)])
    own_at = s["lens"][:, None, None] - n + torch.arange(n, device=DEV)[:, None]
    sees = (t <= own_at) & ((t < c["n_sink"]) | (t > own_at - c["window"]))  # [B, n, T]
    q = s["q"].float().view(B, n, H, -1, D).permute(0, 2, 3, 1, 4)  # [B, H, g, n, D]
    score = SCALE * (q.reshape(B, H, -1, D) @ k.transpose(-1, -2)).view(B, H, -1, n, t.numel())
    score = torch.where(sees[:, None, None], score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, H, -1, t.numel()) @ v).view(B, H, -1, n, D) / torch.where(total == 0, torch.ones_like(total), total)
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(B, n, c["H_q"], D))
    s["lse"].copy_((top + torch.log(total))[..., 0].permute(0, 3, 1, 2).reshape(B, n, c["H_q"]))
    return s["out"], s["lse"]


def _values(c, x, key):
    """The values that the cache stands for, fp64 [B, H_kv, T_cap, D], from
    the bf16 rows x: visual rows of packed heads go through the quantiser."""
    prot, konly, pack = _heads(c)
    bits, out = c["kb"] if key else c["vb"], x.double()
    if bits < 16:
        for h in pack if key else pack + konly:
            code, s, z = _quantise(x[:, h, c["vs"]:c["ve"]], bits, c["G"])
            g = torch.arange(D, device=DEV) // c["G"]
            out[:, h, c["vs"]:c["ve"]] = code.double() * s.double()[..., g] + z.double()[..., g]
    return out


def _exact_window(c, seed):
    k, v, q, lens = _window_inputs(c, seed)
    K, V, g = _values(c, k, True), _values(c, v, False), c["H_q"] // c["H_kv"]
    out, lse = torch.zeros_like(q, dtype=torch.float64), torch.zeros(q.shape[:3], dtype=torch.float64, device=DEV)
    for b, n in enumerate(lens.tolist()):
        for i in range(c["n_q"]):
            at = n - c["n_q"] + i
            t = [x for x in range(min(c["n_sink"], at + 1))]
            t = torch.tensor(t + list(range(max(len(t), at - c["window"] + 1), at + 1)), device=DEV)
            a = torch.einsum("hgd,htd->hgt", q[b, i].double().view(-1, g, D), K[b][:, t]) * SCALE
            out[b, i] = (torch.softmax(a, -1) @ V[b][:, t]).view(-1, D)
            lse[b, i] = torch.logsumexp(a, -1).view(-1)
    return out, lse


# ---- one pass, what it cannot do without, and its definition in 64 bits ------------------

_make = {"rope": _prepare_rope, "verify": _prepare_verify, "window": _prepare_window}
_run_own = {"rope": _own_rope, "verify": _own_verify, "window": _own_window}
_run_plain = {"rope": _plain_rope, "verify": _plain_verify, "window": _plain_window}
_run_exact = {"rope": _exact_rope, "verify": _exact_verify, "window": _exact_window}


def prepare(case, seed):
    return _make[case["op"]](dict(case), seed)


def run(state):
    c = state["c"]
    return (_run_own if own else _run_plain)[c["op"]](c, state)


def exact(case, seed):
    return _run_exact[case["op"]](dict(case), seed)


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
    if c["op"] == "rope":
        rows = c["B"] * c["n"] * (c["H_q"] + c["H_kv"])
        return {"bytes": 4 * D * rows + 4 * c["B"] * c["n"] * len(_ints(c["axes"])) + 2 * c["R"], "flops": 0}
    if c["op"] == "verify":  # rows: logits rows that a sequence's walk visits, the mean over seeds; the draft's where one was turned down
        B, V = c["B"], c["V"]
        row = V * ((2 if c["half"] else 4) * c["rows"] + (4 if c["probs"] else 0) + 4)
        return {"bytes": int(B * (row + 24 * c["n_q"])), "flops": 0}
    total, visual = 0, 0
    for n in _lengths(c):
        first = min(c["n_sink"], n)
        lo = max(first, n - c["n_q"] + 1 - c["window"])
        total += first + n - lo
        visual += sum(max(0, min(b, c["ve"]) - max(a, c["vs"])) for a, b in ((0, first), (lo, n)))
    rows = sum(visual * _row_bytes(c, True, key) + (total - visual) * _row_bytes(c, False, key) for key in (True, False))
    return {"bytes": rows + c["B"] * c["n_q"] * c["H_q"] * (4 * D + 4), "flops": 4 * D * c["H_q"] * c["n_q"] * total}
