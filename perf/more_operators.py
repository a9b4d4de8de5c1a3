"""A chunk of new tokens over a paged KV cache, measured operator by operator.

Three operators, told apart by a case's "op":

  rotate  rotary positions of the heads of a projection's output (both layouts, part of the head,
          frequencies scaled for long contexts, and the transposed rotation, which takes gradients back);
  append  the same rotation of q and K on the way from the projection to the attention's q and to the
          paged cache, V beside it: 16-bit caches, and e4m3 codes with block scales;
  chunk   attention of each sequence's new tokens over its cached rows: causal, in a sliding window,
          or with the drafted tokens' own tree of who sees whom; 16-bit and e4m3 caches.

Every operator has a plain form here in elementary torch operations (`own` false) and the call of
this package that does the same (`own` true).
"""
import math

import torch

own = False

MIN_EXP = -96                        # exponents of block scales are at least this
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "f8": 1}


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # q and K heads of one decode step of a batch of 64, heads of one projection side by side
        dict(name="rotate_step", op="rotate", batch=64, hq=32, hkv=8, d=128, rot=128, layout="half", scaling="plain", dtype="bf16",
             lo=0, hi=8191, new_lo=1, new_hi=1, transposed=False),
        # prompts, half of each head rotated, interleaved pairs, positions scaled linearly
        dict(name="rotate_prompts", op="rotate", batch=16, hq=32, hkv=8, d=128, rot=64, layout="interleaved", scaling="linear", dtype="f16",
             lo=0, hi=0, new_lo=1, new_hi=4096, transposed=False),
        # one decode step of the benchmark's serving shape, far positions, scaled by wavelength
        dict(name="append_step", op="append", batch=16, hq=32, hkv=8, d=128, bs=16, rot=128, layout="half", scaling="wavelength",
             dtype="bf16", kv="bf16", lo=100, hi=131000, new_lo=1, new_hi=1, pad=0),
        # ragged prompts' bulk write
        dict(name="append_prompts", op="append", batch=32, hq=32, hkv=8, d=128, bs=16, rot=128, layout="half", scaling="parts",
             dtype="f16", kv="f16", lo=0, hi=100, new_lo=1, new_hi=2048, pad=0),
        # one decode step of a batch of 128 into an 8-bit cache: single rows, where a block's scale may grow
        dict(name="append_f8_step", op="append", batch=128, hq=32, hkv=8, d=128, bs=16, rot=128, layout="half", scaling="plain",
             dtype="bf16", kv="f8", lo=0, hi=8191, new_lo=1, new_hi=1, pad=0),
        # long ragged prompts into an 8-bit cache
        dict(name="append_f8_prompts", op="append", batch=16, hq=64, hkv=8, d=128, bs=16, rot=64, layout="interleaved", scaling="parts",
             dtype="f16", kv="f8", lo=0, hi=100, new_lo=1, new_hi=4096, pad=3),
        # eight drafted tokens a sequence, a tree of drafts, the benchmark's serving shape
        dict(name="chunk_draft", op="chunk", batch=16, hq=32, hkv=8, d=128, bs=16, dtype="bf16", kv="bf16", lo=4096, hi=4096,
             new_lo=8, new_hi=8, window=0, tree=True),
        # one very long context in an 8-bit cache, eight query heads a KV head, a short chunk
        dict(name="chunk_one_131k_f8", op="chunk", batch=1, hq=64, hkv=8, d=128, bs=32, dtype="bf16", kv="f8", lo=131000, hi=131000,
             new_lo=32, new_hi=32, window=0, tree=False),
        # small heads, a ragged batch of requests that each bring a few tokens
        dict(name="chunk_small_heads", op="chunk", batch=64, hq=12, hkv=12, d=64, bs=16, dtype="f16", kv="f16", lo=1, hi=2000,
             new_lo=1, new_hi=48, window=0, tree=False),
        # whole prompts
        dict(name="chunk_prompts", op="chunk", batch=4, hq=32, hkv=8, d=128, bs=16, dtype="bf16", kv="bf16", lo=0, hi=0,
             new_lo=4096, new_hi=4096, window=0, tree=False),
        # prompts continued in pieces over an 8-bit cache
        dict(name="chunk_pieces_f8", op="chunk", batch=8, hq=32, hkv=8, d=128, bs=16, dtype="f16", kv="f8", lo=1000, hi=16384,
             new_lo=256, new_hi=1024, window=0, tree=False),
        # the same in a sliding window
        dict(name="chunk_window", op="chunk", batch=8, hq=32, hkv=8, d=128, bs=16, dtype="bf16", kv="bf16", lo=5000, hi=20000,
             new_lo=100, new_hi=1000, window=4096, tree=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "append", "append", "chunk", "chunk", "chunk"])
    d, dtype = rng.choice([64, 128]), rng.choice(["f16", "bf16"])
    hkv, g = rng.choice([1, 2, 4, 8, 12]), rng.choice([1, 2, 4, 8])
    bs = rng.choice([8, 16, 16, 32, 64])
    if op != "chunk":
        c = dict(op=op, batch=_log(rng, 1, 128), hq=hkv * g, hkv=hkv, d=d, rot=rng.choice([d, d, d // 2, 16, 48]),
                 layout=rng.choice(["half", "interleaved"]), scaling=rng.choice(["plain", "linear", "parts", "wavelength"]),
                 dtype=rng.choice([dtype, dtype, "f32"]), lo=0, hi=rng.choice([0, 1000, 200000]), new_lo=1, new_hi=1)
        rows = max(1, 6000000 // (c["batch"] * (c["hq"] + 2 * hkv) * d))
        c["new_hi"] = rng.choice([1, 5, _log(rng, 1, max(1, 4 * min(rows, 2048)))])
        if op == "rotate":
            return dict(c, transposed=rng.choice([False, True]))
        return dict(c, bs=bs, kv=rng.choice([c["dtype"], "f8"]), pad=rng.choice([0, 0, 1, 7]))
    batch = _log(rng, 1, 64)
    new_hi = _log(rng, 1, 4096)
    # the scores of the whole batch, were they all held at once
    hi = _log(rng, 1, max(1, min(131072, 1500000000 // (batch * hkv * g * new_hi) - new_hi, 3800000 // (hkv * batch) - new_hi)))
    new_hi = min(new_hi, max(1, 3800000 // (hkv * batch)), max(1, 1500000000 // (batch * hkv * g * new_hi)))
    tree = new_hi <= 64 and rng.random() < 0.4
    return dict(op=op, batch=batch, hq=hkv * g, hkv=hkv, d=d, bs=bs, dtype=dtype, kv=rng.choice([dtype, "f8"]), lo=rng.choice([0, 0, hi]), hi=hi,
                new_lo=rng.choice([0, 1, new_hi]), new_hi=new_hi, window=0 if tree else rng.choice([0, 0, _log(rng, 1, 8192)]), tree=tree)


# ------------------------------------------------------------------------------------ inputs
def _lens(case, seed, lo, hi):
    """A length for each sequence: a case's lengths are the same for every seed, in another order."""
    g = torch.Generator().manual_seed(1000003 * lo + hi)
    lens = torch.randint(lo, hi + 1, (case["batch"],), generator=g, dtype=torch.int64)
    return lens[torch.randperm(case["batch"], generator=torch.Generator().manual_seed(seed))]


def _both(case, seed):
    """Cached and new tokens of each sequence; a sequence keeps its pair."""
    lens, new = _lens(case, seed, case["lo"], case["hi"]), _lens(case, seed, case["new_lo"], case["new_hi"])
    if int(new.sum()) == 0:
        new[0] = 1
    return lens, new


def _rand(shape, gen, dtype, scale=1.0):
    """Normal values, one in a hundred of them eight times larger (keys and values have outliers)."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    big = torch.rand(shape, generator=gen, device="cuda", dtype=torch.float32) < 0.01
    return torch.where(big, x * (8.0 * scale), x * scale).to(dtype)


def _pow2(e):
    """2^e as float32, exactly (-126 <= e <= 127)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _exponent(amax):
    """The least e >= MIN_EXP with amax <= 448 * 2^e = 0.875 * 2^(9 + e), elementwise."""
    m, x = torch.frexp(amax)                              # amax = m * 2^x, m in [0.5, 1)
    e = x - 9 + (m > 0.875).to(x.dtype)
    return torch.where(amax > 0, e.clamp_min(MIN_EXP), torch.full_like(e, MIN_EXP)).to(torch.int32)


def _tables(case, seed, tokens):
    """A random placement of every sequence's blocks: tables [B, most], blocks in the pool."""
    blocks = (tokens + case["bs"] - 1) // case["bs"]
    most, total = max(1, int(blocks.max())), int(blocks.sum())
    nb = total + max(4, total // 16)
    order = torch.randperm(nb, generator=torch.Generator().manual_seed(seed + 7))
    bt = torch.zeros(case["batch"], most, dtype=torch.int32)
    bt[torch.arange(most)[None, :] < blocks[:, None]] = order[:total].to(torch.int32)
    return bt, nb


def _pack(x):
    """Blocks [NB, Hkv, bs, D] -> their e4m3 codes and scales [NB, Hkv]."""
    e = _exponent(x.abs().amax(dim=(2, 3)))
    return (x * _pow2(-e)[:, :, None, None]).to(torch.float8_e4m3fn), _pow2(e)


def _cache(nb, H, bs, D, kv, gen, scale):
    """A cache of `nb` blocks and its scales (None: 16 or 32 bits)."""
    parts, scales = [], []
    for n in range(0, nb, 4096):
        x = _rand((min(4096, nb - n), H, bs, D), gen, torch.float32, scale)
        x, s = _pack(x) if kv == "f8" else (x.to(DTYPES[kv]), None)
        parts.append(x.view(torch.uint8) if kv == "f8" else x)
        scales.append(s)
    return (torch.cat(parts).view(torch.float8_e4m3fn), torch.cat(scales)) if kv == "f8" else (torch.cat(parts), None)


# what a model's configuration says of its positions: base, factor, trained length, and the two limits
ROPE = {"plain": (10000.0, 1.0, 0, 0.0, 0.0), "linear": (10000.0, 4.0, 0, 0.0, 0.0), "parts": (10000.0, 16.0, 4096, 1.0, 32.0),
        "wavelength": (500000.0, 8.0, 8192, 1.0, 4.0)}


def _frequencies(case):
    """Radians a position for each pair of channels, float64, and the factor on the rotated values."""
    base, factor, trained, low, high = ROPE[case["scaling"]]
    r = case["rot"]
    f = base ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] == "parts":                        # pairs of many turns keep theirs, those of few are slowed
        at = lambda turns: r * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        first, last = max(0, math.floor(at(high))), min(r - 1, math.ceil(at(low)))
        slow = ((torch.arange(r // 2, dtype=torch.float64) - first) / max(last - first, 0.001)).clamp(0, 1)
        return f / factor * slow + f * (1 - slow), 0.1 * math.log(factor) + 1.0
    if case["scaling"] == "wavelength":
        keep = ((trained * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        return f / factor * (1 - keep) + f * keep, 1.0
    return f, 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = _prepare_chunk(case, seed, gen) if case["op"] == "chunk" else _prepare_rows(case, seed, gen)
    st["case"] = case
    if own:
        _handles(case, st)
    return st


def _prepare_rows(case, seed, gen):
    B, hq, H, D = case["batch"], case["hq"], case["hkv"], case["d"]
    lens, new = _both(case, seed)
    T = int(new.sum())
    seq = torch.repeat_interleave(torch.arange(B), new)
    nth = torch.arange(T) - torch.repeat_interleave(torch.cumsum(new, 0) - new, new)
    # the output of one projection: a token's q, K and V heads side by side
    qkv = _rand((T, hq + 2 * H, D), gen, DTYPES[case["dtype"]])
    st = dict(qkv=qkv, q=qkv[:, :hq], k=qkv[:, hq:hq + H], v=qkv[:, hq + H:], positions=(lens[seq] + nth).to(torch.int32).cuda())
    f, st["magnitude"] = _frequencies(case)
    st["freqs"] = f.cuda()
    if case["op"] == "rotate":
        st["out"] = torch.zeros(T, hq + H, D, dtype=qkv.dtype, device="cuda")
        return st
    # only the blocks that the step touches need be there: the block of each sequence's next row
    # and the ones after it
    bs = case["bs"]
    start = lens % bs
    bt, st["nb"] = _tables(case, seed, start + new)
    pos = nth + start[seq]
    slots = bt[seq, pos // bs].to(torch.int64) * bs + pos % bs
    if case["pad"]:                                       # a step of fixed capacity ends in padding tokens
        slots[max(1, T - case["pad"]):] = -1
    st["slots"] = slots.to(torch.int32).cuda()
    st["q_out"] = torch.zeros(T, hq, D, dtype=qkv.dtype, device="cuda")
    st["k_cache"], st["k_scales"] = _cache(st["nb"], H, bs, D, case["kv"], gen, 0.25)
    st["v_cache"], st["v_scales"] = _cache(st["nb"], H, bs, D, case["kv"], gen, 0.25)
    return st


def _drafts(new, seed):
    """A random tree over each sequence's new tokens: bit j of token i's word: i descends from j, or is it."""
    g = torch.Generator().manual_seed(seed + 3)
    words = []
    for n in new.tolist():
        parent = (torch.rand(n, generator=g) * (torch.arange(n) + 1)).long() - 1      # -1: a root
        mine = []
        for i, p in enumerate(parent.tolist()):
            mine.append((mine[p] if p >= 0 else 0) | 1 << i)
        words += [w - (1 << 64) if w >> 63 else w for w in mine]
    return torch.tensor(words, dtype=torch.int64).cuda()


def _prepare_chunk(case, seed, gen):
    B, H, D = case["batch"], case["hkv"], case["d"]
    cached, new = _both(case, seed)
    lens = cached + new
    bt, nb = _tables(case, seed, lens)
    T = int(new.sum())
    st = dict(nb=nb, lens=lens.to(torch.int32).cuda(), block_tables=bt.cuda(), max_q_len=max(1, case["new_hi"]), scale=1.0 / math.sqrt(D),
              q_start=torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(new, 0)]).to(torch.int32).cuda(),
              visible=_drafts(new, seed) if case["tree"] else None)
    st["k_cache"], st["k_scales"] = _cache(nb, H, case["bs"], D, case["kv"], gen, 0.6)
    st["v_cache"], st["v_scales"] = _cache(nb, H, case["bs"], D, case["kv"], gen, 0.6)
    st["q"] = (torch.randn((T, case["hq"], D), generator=gen, device="cuda") * 1.5).to(DTYPES[case["dtype"]])
    st["out"] = torch.zeros_like(st["q"])
    return st


def _handles(case, st):
    """What a serving program sets up once: the pool's handle, the rotation's table and the workspace."""
    from paged_kv_cache_273_gb300 import pkv
    if case["op"] != "chunk":
        base, factor, trained, low, high = ROPE[case["scaling"]]
        st["rope"] = pkv.rope_plan(case["rot"], base=base, layout=case["layout"], scaling=case["scaling"], factor=factor, trained_len=trained,
                                   low=low, high=high)
    if case["op"] != "rotate":
        kv = {"f8": pkv.PKV_F8, "f32": pkv.PKV_F32, "f16": pkv.PKV_F16, "bf16": pkv.PKV_BF16}[case["kv"]]
        st["pool"] = pkv.kv_block_pool_init(st["nb"], case["bs"], case["hkv"], case["d"], kv)
    if case["op"] == "chunk":
        st["workspace"] = pkv.alloc_chunk_workspace(st["pool"], case["batch"], case["hq"], st["max_q_len"])


# ------------------------------------------------------------------------------------- calls
def run(st):
    op = st["case"]["op"]
    return _own(st, op) if own else PLAIN[op](st)


def _own(st, op):
    from paged_kv_cache_273_gb300 import pkv
    if op == "rotate":
        hk = st["out"].shape[1]                           # q's and K's heads are side by side: one call
        pkv.kv_rope_rotate(st["rope"], st["qkv"][:, :hk], st["positions"], st["out"], transposed=st["case"]["transposed"])
        return {"out": st["out"]}
    if op == "append":
        pkv.kv_rope_append(st["pool"], st["rope"], st["q"], st["k"], st["v"], st["positions"], st["slots"], st["q_out"], st["k_cache"], st["v_cache"],
                           st["k_scales"], st["v_scales"])
        return _written(st)
    pkv.paged_chunk_attention(st["pool"], st["q"], st["k_cache"], st["v_cache"], st["block_tables"], st["q_start"], st["lens"], st["scale"], st["out"],
                              st["workspace"], st["max_q_len"], st["k_scales"], st["v_scales"], window=st["case"]["window"], visible=st["visible"])
    return {"out": st["out"]}


def _written(st):
    res = {"q": st["q_out"], "k": st["k_cache"], "v": st["v_cache"]}
    if st["k_scales"] is not None:
        res.update(ks=st["k_scales"], vs=st["v_scales"])
    return res


# ------------------------------------------------------------------------------- plain forms
def _rotated(st, x, transposed=False):
    """x [T, H, D] as float32, the first channels of each head rotated."""
    x, r = x.float(), st["case"]["rot"]
    angle = st["positions"].double()[:, None] * st["freqs"]
    c = (torch.cos(angle) * st["magnitude"]).float()[:, None, :]
    s = (torch.sin(angle) * st["magnitude"]).float()[:, None, :]
    if transposed:
        s = -s
    y = x.clone()
    if st["case"]["layout"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2], y[..., r // 2:r] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * c - b * s, b * c + a * s
    return y


def _plain_rotate(st):
    return {"out": _rotated(st, st["qkv"][:, :st["out"].shape[1]], st["case"]["transposed"]).to(st["out"].dtype)}


def _plain_append(st):
    bs = st["case"]["bs"]
    live = st["slots"] >= 0
    slots = st["slots"].long()[live]
    st["q_out"][live] = _rotated(st, st["q"]).to(st["q_out"].dtype)[live]
    for what, x in (("k", _rotated(st, st["k"])[live]), ("v", st["v"].float()[live])):
        if st[what + "_scales"] is None:
            st[what + "_cache"][slots // bs, :, slots % bs] = x.to(st[what + "_cache"].dtype)
        else:
            _plain_codes(st[what + "_cache"], st[what + "_scales"], x, slots, bs)
    return _written(st)


def _plain_codes(cache, scales, x, slots, bs):
    """New rows x [T, H, D] into a cache of e4m3 codes; a block's scale grows with its rows."""
    ids, at = torch.unique(slots // bs, return_inverse=True)
    start = torch.full((ids.numel(),), bs, device="cuda").scatter_reduce(0, at, slots % bs, "amin")
    T, H, _ = x.shape
    e_new = _exponent(torch.zeros(ids.numel(), H, device="cuda").scatter_reduce(0, at[:, None].expand(T, H), x.abs().amax(dim=2), "amax"))
    e_old = (((scales[ids].view(torch.int32) >> 23) & 255) - 127).clamp_min(MIN_EXP)
    e = torch.where((start == 0)[:, None], e_new, torch.maximum(e_old, e_new))
    # rows before the first new one, at the block's new scale
    codes = cache.view(torch.uint8)
    held = codes[ids].view(torch.float8_e4m3fn)
    again = (held.float() * _pow2((e_old - e).clamp(-126, 0))[:, :, None, None]).to(torch.float8_e4m3fn)
    keep = torch.arange(bs, device="cuda")[None, :] < start[:, None]
    codes[ids] = torch.where(keep[:, None, :, None], again.view(torch.uint8), held.view(torch.uint8))
    codes[ids[at], :, slots % bs] = (x * _pow2(-e)[at][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    scales[ids] = _pow2(e)


def _held(cache, scales, ids):
    """Blocks `ids` [B, n] of a cache as float32 rows [B, Hkv, n * bs, D]."""
    x = cache[ids].float() if scales is None else cache.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float() * scales[ids][..., None, None]
    B, n, H, bs, D = x.shape
    return x.transpose(1, 2).reshape(B, H, n * bs, D)


def _plain_chunk(st):
    c = st["case"]
    B, H, D, G, n = c["batch"], c["hkv"], c["d"], c["hq"] // c["hkv"], st["max_q_len"]
    T, ids, lens, start = st["q"].shape[0], st["block_tables"].long(), st["lens"].long(), st["q_start"].long()
    new, i = start[1:] - start[:-1], torch.arange(n, device="cuda")
    # every sequence's new tokens side by side, as many as the longest has
    rows = (start[:-1, None] + i).clamp_max(T - 1)
    q = st["q"].float()[rows].view(B, n, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * n, D)
    s = (q @ _held(st["k_cache"], st["k_scales"], ids).transpose(-1, -2)) * st["scale"]
    key = torch.arange(s.shape[-1], device="cuda")
    at = (lens - new)[:, None] + i                        # positions [B, n]
    sees = key <= at[..., None]
    if c["window"]:
        sees &= key > at[..., None] - c["window"]
    if c["tree"]:
        j = key - (lens - new)[:, None]                   # [B, keys]: which new token a key is
        bit = (st["visible"][rows][..., None] >> j.clamp(0, 63)[:, None, :]) & 1
        sees = (j < 0)[:, None, :] | ((bit != 0) & (j < new[:, None])[:, None, :])
    s = s.view(B, H, G, n, -1).masked_fill(~sees[:, None, None], -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    den = p.sum(dim=-1, keepdim=True)
    o = p.view(B, H, G * n, -1) @ _held(st["v_cache"], st["v_scales"], ids)
    o = (o.view(B, H, G, n, D) / torch.where(den > 0, den, 1.0)).permute(0, 3, 1, 2, 4).reshape(B, n, H * G, D)
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(start[1:], t, right=True)
    return {"out": o[b, t - start[b]].to(st["q"].dtype)}


PLAIN = {"rotate": _plain_rotate, "append": _plain_append, "chunk": _plain_chunk}


# -------------------------------------------------------------------------------------- work
def work(case):
    B, hq, H, D = case["batch"], case["hq"], case["hkv"], case["d"]
    mean, new = (case["lo"] + case["hi"]) / 2, (case["new_lo"] + case["new_hi"]) / 2
    if case["op"] == "chunk":
        sees = min(mean + new / 2, case["window"] or math.inf)
        read = min(mean + new, (case["window"] or math.inf) + new)
        return {"bytes": B * (2 * read * H * D * SIZE[case["kv"]] + 2 * new * hq * D * SIZE[case["dtype"]]), "flops": 4 * B * new * sees * hq * D}
    T, eb = B * new, SIZE[case["dtype"]]
    turned = T * (hq + H) * case["rot"]
    if case["op"] == "rotate":
        return {"bytes": 2 * T * (hq + H) * D * eb + 4 * T, "flops": 3 * turned}
    return {"bytes": T * ((2 * hq + 2 * H) * D * eb + 2 * H * D * SIZE[case["kv"]] + 8), "flops": 3 * turned}


# --------------------------------------------------------------------------- 64-bit definition
def exact(case, seed):
    """The operators' outputs from their definitions, in float64."""
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "chunk":
        return _exact_chunk(st)
    if case["op"] == "rotate":
        return {"out": _exact_turn(st, st["qkv"][:, :st["out"].shape[1]], case["transposed"])}
    return _exact_append(st)


def _exact_turn(st, x, back=False):
    """Pairs of channels as complex numbers, times m e^(i p theta)."""
    r, half = st["case"]["rot"], st["case"]["layout"] == "half"
    x = x.double()
    turn = torch.polar(torch.full((1,), st["magnitude"], dtype=torch.float64, device="cuda"), st["positions"].double()[:, None] * st["freqs"])
    if back:
        turn = turn.conj()
    head = x[..., :r]
    pairs = head.unflatten(-1, (2, r // 2)).transpose(-1, -2) if half else head.unflatten(-1, (r // 2, 2))
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None, :])
    return torch.cat([(z.transpose(-1, -2) if half else z).flatten(-2), x[..., r:]], dim=-1)


def _e4m3(x):
    """float64 values -> the nearest e4m3 values (ties to even), |x| <= 448."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 4).clamp_min(-9).double())     # 4 significant bits; 2^-9 below 2^-6
    return torch.round(x / step) * step


def _exact_append(st):
    bs = st["case"]["bs"]
    ls = st["slots"].tolist()
    live = [t for t in range(len(ls)) if ls[t] >= 0]
    q, at = st["q_out"].double(), torch.tensor(live, device="cuda")
    q[at] = _exact_turn(st, st["q"])[at]
    res = {"q": q}
    to = st["slots"].long()[at]
    rows = {"k": _exact_turn(st, st["k"])[at], "v": st["v"].double()[at]}
    if st["k_scales"] is None:
        for what in "kv":
            res[what] = st[what + "_cache"].double()
            res[what][to // bs, :, to % bs] = rows[what]
        return res
    # runs of consecutive slots inside one block, one after another
    cut = [i for i, t in enumerate(live) if i == 0 or ls[t] != ls[live[i - 1]] + 1 or ls[t] % bs == 0]
    first = torch.tensor(cut)
    run = torch.repeat_interleave(torch.arange(len(cut)), torch.diff(torch.cat([first, torch.tensor([len(live)])]))).cuda()
    block, start = (to[first.cuda()] // bs), (to[first.cuda()] % bs)
    for what in "kv":
        x, codes, scales = rows[what], st[what + "_cache"].double(), st[what + "_scales"].double()
        amax = torch.zeros(len(cut), x.shape[1], dtype=torch.float64, device="cuda").index_reduce_(0, run, x.abs().amax(dim=2), "amax")
        need = torch.where(amax > 0, torch.ceil(torch.log2(amax.clamp_min(1e-300) / 448.0) - 1e-13), torch.full_like(amax, -96.0)).clamp_min(-96.0)
        need = torch.where(amax > 448.0 * torch.exp2(need), need + 1, need)
        s_new, s_old = torch.exp2(need), scales[block]
        s = torch.where((start == 0)[:, None], s_new, torch.maximum(s_old, s_new))
        held = codes[block]
        again = _e4m3(held * (s_old / s).clamp_max(1.0)[:, :, None, None])
        before = torch.arange(bs, device="cuda")[None, :] < start[:, None]
        codes[block] = torch.where(before[:, None, :, None], again, held)
        codes[to // bs, :, to % bs] = _e4m3(x / s[run][:, :, None])
        scales[block] = s
        res[what], res[what + "s"] = codes, scales
    return res


def _exact_chunk(st):
    c = st["case"]
    H, D, bs, G = c["hkv"], c["d"], c["bs"], c["hq"] // c["hkv"]
    lens, start = st["lens"].tolist(), st["q_start"].tolist()
    if 4.0 * sum((start[b + 1] - start[b]) * lens[b] for b in range(len(lens))) * c["hq"] * D > 6e12:
        return None

    def rows(what, ids, h):
        x = st[what + "_cache"]
        if st[what + "_scales"] is None:
            return x[ids, h].double().reshape(-1, D)
        return (x.view(torch.uint8)[ids, h].view(torch.float8_e4m3fn).double() * st[what + "_scales"][ids, h].double()[:, None, None]).reshape(-1, D)

    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for b, L in enumerate(lens):
        n = start[b + 1] - start[b]
        if n == 0:
            continue
        ids = st["block_tables"][b, :-(-L // bs)].long()
        key, pos = torch.arange(L, device="cuda"), torch.arange(L - n, L, device="cuda")[:, None]
        hidden = key > pos
        if c["window"]:
            hidden |= key <= pos - c["window"]
        if c["tree"]:
            words = st["visible"][start[b]:start[b + 1]]
            own_bits = torch.stack([(words >> j) & 1 for j in range(n)], dim=1) == 0
            hidden = torch.cat([torch.zeros(n, L - n, dtype=torch.bool, device="cuda"), own_bits], dim=1)
        for h in range(H):
            k, v = rows("k", ids, h)[:L], rows("v", ids, h)[:L]
            for g in range(h * G, h * G + G):
                s = (st["q"][start[b]:start[b + 1], g].double() @ k.T) * st["scale"]
                out[start[b]:start[b + 1], g] = torch.softmax(s.masked_fill(hidden, -math.inf), dim=1) @ v
    return {"out": out}
