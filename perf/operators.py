"""The device-resident decode step over a paged KV cache, measured operator by operator.

Five operators, told apart by a case's "op":

  tables  block tables, slot mapping and token offsets from request lengths ("reserve"), and the
          blocks of finished sequences back to the free list ("release"), all on the device;
  append  new K and V rows into a cache of e4m3 codes with one power-of-two scale for each
          (block, KV head) of K and of V;
  attend  one query token for each sequence over that cache;
  bounds  the running int8 lower and upper bounds of each block's keys;
  sparse  one query token for each sequence over the blocks that those bounds score highest.

Every operator has a plain form here in elementary torch operations (`own` false) and the call of
this package that does the same (`own` true).
"""
import math

import torch

own = False

BS_MIN_EXP = -96                     # exponents of block scales and bounds are at least this
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "f8": torch.float8_e4m3fn}


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step's bookkeeping of a full serving batch: one new token a sequence
        dict(name="tables_step", op="tables", what="reserve", batch=512, bs=16, lo=0, hi=8192, new_lo=1, new_hi=1),
        # admission of a batch of prompts: nearly a million slots, a block table entry every 16
        dict(name="tables_prompts", op="tables", what="reserve", batch=256, bs=16, lo=0, hi=0, new_lo=1, new_hi=8192),
        # a quarter of a large batch finishes and returns its blocks
        dict(name="tables_release", op="tables", what="release", batch=1024, bs=16, lo=0, hi=4096, new_lo=0, new_hi=0),
        # the append of one decode step: single rows into partly filled blocks, where a scale may grow
        dict(name="append_step", op="append", batch=128, hkv=8, d=128, bs=16, dtype="bf16", lo=0, hi=4095, new_lo=1, new_hi=1),
        # the bulk write of ragged prompts, some of them continuing a partly filled block
        dict(name="append_prompts", op="append", batch=32, hkv=8, d=128, bs=16, dtype="f16", lo=0, hi=100, new_lo=1, new_hi=8192),
        # a single short request on small heads: latency
        dict(name="attend_one", op="attend", batch=1, hq=12, hkv=12, d=64, bs=16, dtype="f16", lo=1000, hi=1000),
        # the benchmark's serving shape
        dict(name="attend_16x4096", op="attend", batch=16, hq=32, hkv=8, d=128, bs=16, dtype="bf16", lo=4096, hi=4096),
        # a large ragged batch
        dict(name="attend_ragged128", op="attend", batch=128, hq=32, hkv=8, d=128, bs=16, dtype="f16", lo=512, hi=8192),
        # the key bounds of one decode step's rows
        dict(name="bounds_step", op="bounds", batch=128, hkv=8, d=128, bs=16, dtype="bf16", lo=0, hi=4095, new_lo=1, new_hi=1),
        # the key bounds of ragged prompts
        dict(name="bounds_prompts", op="bounds", batch=32, hkv=8, d=128, bs=16, dtype="f16", lo=0, hi=100, new_lo=1, new_hi=8192),
        # long contexts, a sixteenth of each attended
        dict(name="sparse_16x32k", op="sparse", batch=16, hq=32, hkv=8, d=128, bs=16, dtype="bf16", kv="bf16", lo=32000, hi=32768, budget=128),
        # one very long context over the 8-bit cache, eight query heads a KV head
        dict(name="sparse_one_131k", op="sparse", batch=1, hq=64, hkv=8, d=128, bs=32, dtype="bf16", kv="f8", lo=131001, hi=131072, budget=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "attend", "attend", "bounds", "sparse", "sparse"])
    bs = rng.choice([8, 16, 16, 32, 64])
    if op == "tables":
        what = rng.choice(["reserve", "reserve", "release"])
        batch = _log(rng, 1, 1024)
        hi = _log(rng, 1, min(16384, max(1, 1000000 // batch)))
        if what == "release":
            return dict(op=op, what=what, batch=batch, bs=bs, lo=0, hi=hi, new_lo=0, new_hi=0)
        new_hi = rng.choice([1, 7, _log(rng, 1, min(8192, max(1, 1000000 // batch)))])
        return dict(op=op, what=what, batch=batch, bs=bs, lo=0, hi=hi, new_lo=min(1, rng.randrange(2)), new_hi=new_hi)
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8, 12])
    g = rng.choice([1, 2, 4, 8])
    dtype = rng.choice(["f16", "bf16"])
    if op in ("append", "bounds"):
        batch = _log(rng, 1, 256)
        new_hi = rng.choice([1, 5, _log(rng, 1, min(8192, max(1, 1000000 // (hkv * batch))))])
        return dict(op=op, batch=batch, hkv=hkv, d=d, bs=bs, dtype=rng.choice([dtype, dtype, "f32"]), lo=0, hi=_log(rng, 1, 2048),
                    new_lo=1, new_hi=new_hi)
    if op == "attend":
        batch = _log(rng, 1, 128)
        hi = _log(rng, 17, max(17, min(16384, 4000000 // (hkv * batch))))
        return dict(op=op, batch=batch, hq=hkv * g, hkv=hkv, d=d, bs=bs, dtype=dtype, lo=rng.choice([0, 1, hi]), hi=hi)
    batch = _log(rng, 1, 32)
    hi = _log(rng, 100, max(100, min(131072, 4000000 // (hkv * batch))))
    return dict(op=op, batch=batch, hq=hkv * g, hkv=hkv, d=d, bs=bs, dtype=dtype, kv=rng.choice([dtype, "f8"]),
                lo=rng.choice([1, max(1, hi - 50)]), hi=hi, budget=rng.choice([1, 8, 33, 64, 128]))


# ------------------------------------------------------------------------------------ inputs
def _lens(case, seed, lo, hi):
    """A length for each sequence: a case's lengths are the same for every seed, in another order."""
    g = torch.Generator().manual_seed(1000003 * lo + hi)
    lens = torch.randint(lo, hi + 1, (case["batch"],), generator=g, dtype=torch.int64)
    return lens[torch.randperm(case["batch"], generator=torch.Generator().manual_seed(seed))]


def _rand(shape, gen, dtype, scale=1.0):
    """Normal values, one in a hundred of them eight times larger (keys and values have outliers)."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    big = torch.rand(shape, generator=gen, device="cuda", dtype=torch.float32) < 0.01
    return torch.where(big, x * (8.0 * scale), x * scale).to(dtype)


def _pow2(e):
    """2^e as float32, exactly (-126 <= e <= 127)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _exponent(amax, top_mantissa, top_exponent):
    """The least e >= BS_MIN_EXP with amax <= top_mantissa * 2^(top_exponent + e), elementwise."""
    m, x = torch.frexp(amax)                              # amax = m * 2^x, m in [0.5, 1)
    e = x - top_exponent + (m > top_mantissa).to(x.dtype)
    return torch.where(amax > 0, e.clamp_min(BS_MIN_EXP), torch.full_like(e, BS_MIN_EXP)).to(torch.int32)


def _exp_codes(amax):
    return _exponent(amax, 0.875, 9)                      # 448 = 0.875 * 2^9


def _exp_bounds(amax):
    return _exponent(amax, 0.9921875, 7)                  # 127 = 0.9921875 * 2^7


def _tables(case, seed, tokens):
    """A random placement of every sequence's blocks: tables [B, most], blocks in the pool."""
    blocks = (tokens + case["bs"] - 1) // case["bs"]
    most = max(1, int(blocks.max()))
    total = int(blocks.sum())
    nb = total + max(4, total // 16)
    g = torch.Generator().manual_seed(seed + 7)
    order = torch.randperm(nb, generator=g)
    bt = torch.zeros(case["batch"], most, dtype=torch.int32)
    held = torch.arange(most)[None, :] < blocks[:, None]
    bt[held] = order[:total].to(torch.int32)
    return bt, nb, order[total:], blocks


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op == "tables":
        st = _prepare_tables(case, seed)
    elif op in ("append", "bounds"):
        st = _prepare_rows(case, seed, gen)
    else:
        st = _prepare_attend(case, seed, gen)
    st["case"] = case
    if own:
        _handles(case, st)
    return st


def _prepare_tables(case, seed):
    B, bs = case["batch"], case["bs"]
    lens = _lens(case, seed, case["lo"], case["hi"])
    new = _lens(case, seed, case["new_lo"], case["new_hi"])   # a sequence keeps its pair of lengths
    old = (lens + bs - 1) // bs
    need = (lens + new + bs - 1) // bs
    most = max(1, int(need.max()))
    nb = int(need.sum()) + 8
    g = torch.Generator().manual_seed(seed + 2)
    order = torch.randperm(nb, generator=g).to(torch.int32)
    bt = torch.zeros(B, most, dtype=torch.int32)
    bt[torch.arange(most)[None, :] < old[:, None]] = order[:int(old.sum())]
    free = order[int(old.sum()):]
    free_ids = torch.zeros(nb, dtype=torch.int32)
    free_ids[:free.numel()] = free
    done = (torch.randperm(B, generator=g) < B // 4).to(torch.int32)
    dev = lambda t: t.to(torch.int32).cuda()  # noqa: E731
    st = dict(nb=nb, free_ids=free_ids.cuda(), free_in=torch.tensor([free.numel(), 0], dtype=torch.int32).cuda(),
              free_out=torch.zeros(2, dtype=torch.int32, device="cuda"), lens=dev(lens), lens_out=torch.zeros(B, dtype=torch.int32, device="cuda"),
              new=dev(new), block_tables=bt.cuda(), done=done.cuda())
    # a serving loop's slot buffer has a fixed capacity; entries past the tokens are padding
    st["slots"] = torch.zeros(max(1, B * case["new_hi"] if case["new_hi"] <= 16 else int(new.sum()) + 64), dtype=torch.int32, device="cuda")
    st["q_start"] = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    return st


def _prepare_rows(case, seed, gen):
    B, bs, H, D = case["batch"], case["bs"], case["hkv"], case["d"]
    lens = _lens(case, seed, case["lo"], case["hi"])
    new = _lens(case, seed, case["new_lo"], case["new_hi"])   # a sequence keeps its pair of lengths
    # only the blocks that the step touches need be there: the block of each sequence's next row
    # and the ones after it
    start = lens % bs
    bt, nb, _, _ = _tables(case, seed, start + new)
    T = int(new.sum())
    seq = torch.repeat_interleave(torch.arange(B), new)
    pos = torch.arange(T) - torch.repeat_interleave(torch.cumsum(new, 0) - new, new) + start[seq]
    slots = bt[seq, pos // bs].to(torch.int64) * bs + pos % bs
    st = dict(nb=nb, slots=slots.to(torch.int32).cuda(), k_new=_rand((T, H, D), gen, DTYPES[case["dtype"]]),
              v_new=_rand((T, H, D), gen, DTYPES[case["dtype"]]))
    if case["op"] == "append":
        st["k_cache"], st["k_scales"] = _pack(_rand((nb, H, bs, D), gen, torch.float32, 0.25))
        st["v_cache"], st["v_scales"] = _pack(_rand((nb, H, bs, D), gen, torch.float32, 0.25))
    else:
        st["bounds"], st["bound_exps"] = _bound(_rand((nb, H, bs, D), gen, torch.float32, 0.25))
    return st


def _pack(x):
    """Blocks [NB, Hkv, bs, D] -> their e4m3 codes and scales [NB, Hkv]."""
    e = _exp_codes(x.abs().amax(dim=(2, 3)))
    return (x * _pow2(-e)[:, :, None, None]).to(torch.float8_e4m3fn), _pow2(e)


def _bound(x):
    """Blocks of keys [NB, Hkv, bs, D] -> int8 bounds [NB, Hkv, 2, D] and exponents [NB, Hkv]."""
    lo, hi = x.amin(dim=2), x.amax(dim=2)
    e = _exp_bounds(torch.maximum(lo.abs(), hi.abs()).amax(dim=2))
    f = _pow2(-e)[:, :, None]
    return torch.stack([torch.floor(lo * f), torch.ceil(hi * f)], dim=2).to(torch.int8), e


def _prepare_attend(case, seed, gen):
    B, H, D, bs = case["batch"], case["hkv"], case["d"], case["bs"]
    lens = _lens(case, seed, case["lo"], case["hi"])
    bt, nb, _, _ = _tables(case, seed, lens)
    sparse = case["op"] == "sparse"
    st = dict(nb=nb, lens=lens.to(torch.int32).cuda(), block_tables=bt.cuda(), max_seq_len=case["hi"], scale=1.0 / math.sqrt(D))
    kv = case.get("kv", "f8")
    caches = []
    for what in "kv":
        parts, scales = [], []
        for n in range(0, nb, 4096):
            m = min(4096, nb - n)
            x = _rand((m, H, bs, D), gen, torch.float32, 0.6)
            if sparse and what == "k":                    # neighbouring tokens have keys in common
                x += torch.randn((m, H, 1, D), generator=gen, device="cuda") * 0.8
                if kv != "f8":
                    x = x.to(DTYPES[kv]).float()
                b, e = _bound(x)
                st.setdefault("bounds", []).append(b)
                st.setdefault("bound_exps", []).append(e)
            if kv == "f8":
                x, s = _pack(x)
                parts.append(x.view(torch.uint8))
                scales.append(s)
            else:
                parts.append(x.to(DTYPES[kv]))
        c = torch.cat(parts)
        caches.append((c.view(torch.float8_e4m3fn), torch.cat(scales)) if kv == "f8" else (c, None))
    (st["k_cache"], st["k_scales"]), (st["v_cache"], st["v_scales"]) = caches
    if sparse:
        st["bounds"], st["bound_exps"] = torch.cat(st["bounds"]), torch.cat(st["bound_exps"])
        st["selected"] = torch.zeros(B, H, case["budget"], dtype=torch.int32, device="cuda")
    st["q"] = (torch.randn((B, case["hq"], D), generator=gen, device="cuda") * 1.5).to(DTYPES[case["dtype"]])
    st["out"] = torch.zeros(B, case["hq"], D, dtype=torch.float32, device="cuda")
    return st


def _handles(case, st):
    """What a serving program sets up once: the pool's handle and the workspaces."""
    from paged_kv_cache_273_gb300 import pkv
    kv = {"f8": pkv.PKV_F8, "f16": pkv.PKV_F16, "bf16": pkv.PKV_BF16}[case.get("kv", "f8")]
    st["pool"] = pkv.kv_block_pool_init(st["nb"], case["bs"], case.get("hkv", 1), case.get("d", 128), kv)
    if case["op"] == "attend":
        st["workspace"] = pkv.alloc_workspace(st["pool"], case["batch"], case["hq"])
    if case["op"] == "sparse":
        st["workspace"] = pkv.alloc_sparse_workspace(st["pool"], case["batch"], case["hq"], case["hi"], case["budget"])


# ------------------------------------------------------------------------------------- calls
def run(st):
    op = st["case"]["op"]
    return _own(st, op) if own else PLAIN[op](st)


def _own(st, op):
    from paged_kv_cache_273_gb300 import pkv
    if op == "tables" and st["case"]["what"] == "reserve":
        pkv.kv_device_reserve(st["pool"], st["free_ids"], st["free_in"], st["lens"], st["block_tables"], st["slots"],
                              num_new=st["new"], free_out=st["free_out"], seq_lens_out=st["lens_out"], q_start=st["q_start"])
        return {"slots": st["slots"], "tables": st["block_tables"], "lens": st["lens_out"], "q_start": st["q_start"], "free": st["free_out"][:1]}
    if op == "tables":
        pkv.kv_device_release(st["pool"], st["free_ids"], st["free_in"], st["lens"], st["done"], st["block_tables"],
                              free_out=st["free_out"], seq_lens_out=st["lens_out"])
        return {"free_ids": st["free_ids"], "lens": st["lens_out"], "free": st["free_out"][:1]}
    if op == "append":
        pkv.kv_append(st["pool"], st["k_new"], st["v_new"], st["slots"], st["k_cache"], st["v_cache"], st["k_scales"], st["v_scales"])
        return {"k": st["k_cache"], "v": st["v_cache"], "ks": st["k_scales"], "vs": st["v_scales"]}
    if op == "bounds":
        pkv.kv_bounds_append(st["pool"], st["k_new"], st["slots"], st["bounds"], st["bound_exps"])
        return {"bounds": st["bounds"], "exps": st["bound_exps"]}
    if op == "attend":
        pkv.paged_decode_attention(st["pool"], st["q"], st["k_cache"], st["v_cache"], st["block_tables"], st["lens"], st["scale"], st["out"],
                                   st["workspace"], st["max_seq_len"], st["k_scales"], st["v_scales"])
        return {"out": st["out"]}
    pkv.paged_decode_attention_sparse(st["pool"], st["q"], st["k_cache"], st["v_cache"], st["bounds"], st["bound_exps"], st["block_tables"],
                                      st["lens"], st["scale"], st["out"], st["selected"], st["workspace"], st["max_seq_len"],
                                      st["k_scales"], st["v_scales"])
    return {"out": st["out"], "selected": st["selected"]}


# ------------------------------------------------------------------------------- plain forms
def _plain_tables(st):
    c = st["case"]
    bs, lens, bt = c["bs"], st["lens"].long(), st["block_tables"]
    B, most = bt.shape
    count = st["free_in"][0].long()
    old = (lens + bs - 1) // bs
    if c["what"] == "release":
        gone = (torch.arange(most, device="cuda")[None, :] < old[:, None]) & (st["done"] != 0)[:, None]
        ids = bt[gone]
        st["free_ids"][count + torch.arange(ids.numel(), device="cuda")] = ids
        return {"free_ids": st["free_ids"], "lens": torch.where(st["done"] != 0, 0, lens).to(torch.int32),
                "free": (count + ids.numel()).to(torch.int32).reshape(1)}
    new = st["new"].long()
    grow = (lens + new + bs - 1) // bs - old
    blk = torch.cumsum(grow, 0) - grow
    # table entries: the k-th new block of the batch is the k-th from the top of the free list
    j = torch.arange(most, device="cuda")[None, :] - old[:, None]
    fresh = (j >= 0) & (j < grow[:, None])
    top = (count - 1 - (blk[:, None] + j)).clamp(0, st["nb"] - 1)
    bt.copy_(torch.where(fresh, st["free_ids"][top], bt))
    # slots: one entry for each new token, in sequence order, -1 behind the last
    end = torch.cumsum(new, 0)
    t = torch.arange(st["slots"].numel(), device="cuda")
    b = torch.searchsorted(end, t, right=True).clamp_max(B - 1)
    pos = (lens[b] + t - (end[b] - new[b])).clamp(0, most * bs - 1)
    slots = torch.where(t < end[-1], bt[b, pos // bs].long() * bs + pos % bs, -1)
    q_start = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), end])
    return {"slots": slots.to(torch.int32), "tables": bt, "lens": (lens + new).to(torch.int32), "q_start": q_start.to(torch.int32),
            "free": (count - grow.sum()).to(torch.int32).reshape(1)}


def _touched(st, bs):
    """The blocks that new rows go to, the first offset written in each, and each row's place in that list."""
    slots = st["slots"].long()
    ids, at = torch.unique(slots // bs, return_inverse=True)
    start = torch.full((ids.numel(),), bs, device="cuda").scatter_reduce(0, at, slots % bs, "amin")
    return slots, ids, at, start


def _plain_append(st):
    bs = st["case"]["bs"]
    slots, ids, at, start = _touched(st, bs)
    res = {}
    for what, new in (("k", st["k_new"]), ("v", st["v_new"])):
        cache, scales = st[what + "_cache"], st[what + "_scales"]
        x = new.float()
        T, H, D = x.shape
        amax = torch.zeros(ids.numel(), H, device="cuda").scatter_reduce(0, at[:, None].expand(T, H), x.abs().amax(dim=2), "amax")
        e_new = _exp_codes(amax)
        e_old = ((scales[ids].view(torch.int32) >> 23) & 255) - 127
        e_old = e_old.clamp_min(BS_MIN_EXP)
        e = torch.where((start == 0)[:, None], e_new, torch.maximum(e_old, e_new))
        # rows before the first new one, at the block's new scale
        codes = cache.view(torch.uint8)
        held = codes[ids].view(torch.float8_e4m3fn)
        again = (held.float() * _pow2((e_old - e).clamp(-126, 0))[:, :, None, None]).to(torch.float8_e4m3fn)
        keep = torch.arange(bs, device="cuda")[None, :] < start[:, None]
        codes[ids] = torch.where(keep[:, None, :, None], again.view(torch.uint8), held.view(torch.uint8))
        # the new rows
        codes[ids[at], :, slots % bs] = (x * _pow2(-e)[at][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[ids] = _pow2(e)
        res[what], res[what + "s"] = cache, scales
    return res


def _plain_bounds(st):
    bs, bounds, exps = st["case"]["bs"], st["bounds"], st["bound_exps"]
    _, ids, at, start = _touched(st, bs)
    x = st["k_new"].float()
    T, H, D = x.shape
    to = at[:, None, None].expand(T, H, D)
    lo = torch.full((ids.numel(), H, D), math.inf, device="cuda").scatter_reduce(0, to, x, "amin")
    hi = torch.full((ids.numel(), H, D), -math.inf, device="cuda").scatter_reduce(0, to, x, "amax")
    e_new = _exp_bounds(torch.maximum(lo.abs(), hi.abs()).amax(dim=2))
    fresh = (start == 0)[:, None]
    e_old = exps[ids].clamp_min(BS_MIN_EXP)
    e = torch.where(fresh, e_new, torch.maximum(e_old, e_new))
    f, down = _pow2(-e)[:, :, None], (e - e_old).clamp(0, 31)[:, :, None]
    lo, hi = torch.floor(lo * f).to(torch.int32), torch.ceil(hi * f).to(torch.int32)
    was = bounds[ids].to(torch.int32)
    lo = torch.where(fresh[:, :, None], lo, torch.minimum(lo, was[:, :, 0] >> down))
    hi = torch.where(fresh[:, :, None], hi, torch.maximum(hi, -((-was[:, :, 1]) >> down)))
    bounds[ids] = torch.stack([lo, hi], dim=2).to(torch.int8)
    exps[ids] = e
    return {"bounds": bounds, "exps": exps}


def _softmax_v(q, k, v, valid, scale):
    """q [.., G, D], k and v [.., n, D], valid [.., n]: masked attention; no valid row gives zeros."""
    s = (q @ k.transpose(-1, -2)) * scale
    s = s.masked_fill(~valid[..., None, :], -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    den = p.sum(dim=-1, keepdim=True)
    return torch.where(den > 0, (p @ v) / den, torch.zeros_like(den))


def _rows(cache, scales, ids):
    """Blocks `ids` of a cache, all heads, as float32: [*ids, Hkv, bs, D]."""
    if scales is None:
        return cache[ids].float()
    return cache.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float() * scales[ids][..., None, None]


def _plain_attend(st):
    c, ids = st["case"], st["block_tables"].long()
    B, n = ids.shape
    H, D, bs = c["hkv"], c["d"], c["bs"]
    k = _rows(st["k_cache"], st["k_scales"], ids).transpose(1, 2).reshape(B, H, n * bs, D)
    v = _rows(st["v_cache"], st["v_scales"], ids).transpose(1, 2).reshape(B, H, n * bs, D)
    q = st["q"].float().view(B, H, -1, D)
    valid = (torch.arange(n * bs, device="cuda")[None, :] < st["lens"][:, None])[:, None, :]
    return {"out": _softmax_v(q, k, v, valid, st["scale"]).reshape(B, c["hq"], D)}


def _plain_sparse(st):
    c, ids = st["case"], st["block_tables"].long()
    B, n = ids.shape
    H, D, bs, budget = c["hkv"], c["d"], c["bs"], c["budget"]
    lens = st["lens"].long()
    nblk = (lens + bs - 1) // bs
    q = st["q"].float().view(B, H, -1, D)
    # whole-number scores: q in steps of a power of two, against the block bounds
    qi = torch.round(q * _pow2(-_exp_bounds(q.abs().amax(dim=(2, 3))))[:, :, None, None])
    bounds = st["bounds"][ids].float()                    # [B, n, H, 2, D]
    up = qi.clamp_min(0) @ bounds[:, :, :, 1].permute(0, 2, 3, 1)
    dn = qi.clamp_max(0) @ bounds[:, :, :, 0].permute(0, 2, 3, 1)
    score = (up + dn).amax(dim=2) * _pow2(st["bound_exps"][ids].clamp_min(BS_MIN_EXP)).transpose(1, 2)
    # the newest block first, then by score, the lower index first among equals
    j = torch.arange(n, device="cuda")
    score = torch.where(j == (nblk - 1)[:, None, None], math.inf, score)
    score = torch.where(j < nblk[:, None, None], score, -math.inf)
    best = torch.sort(score, dim=2, descending=True, stable=True).indices
    take = min(budget, n)
    chosen = best[:, :, :take]
    chosen = torch.where(torch.arange(take, device="cuda") < nblk[:, None, None], chosen, n)
    chosen = torch.sort(chosen, dim=2).values             # ascending, absent ones last
    there = chosen < n
    at = chosen.clamp_max(n - 1)
    phys = ids[torch.arange(B, device="cuda")[:, None, None], at]                  # [B, H, take]
    head = torch.arange(H, device="cuda")[None, :, None]
    k = _chosen_rows(st["k_cache"], st["k_scales"], phys, head).reshape(B, H, take * bs, D)
    v = _chosen_rows(st["v_cache"], st["v_scales"], phys, head).reshape(B, H, take * bs, D)
    pos = at[..., None] * bs + torch.arange(bs, device="cuda")
    valid = (there[..., None] & (pos < lens[:, None, None, None])).reshape(B, H, take * bs)
    out = _softmax_v(q, k, v, valid, st["scale"]).reshape(B, c["hq"], D)
    selected = torch.full((B, H, budget), -1, dtype=torch.int32, device="cuda")
    selected[:, :, :take] = torch.where(there, chosen, -1).to(torch.int32)
    return {"out": out, "selected": selected}


def _chosen_rows(cache, scales, phys, head):
    if scales is None:
        return cache[phys, head].float()
    return cache.view(torch.uint8)[phys, head].view(torch.float8_e4m3fn).float() * scales[phys, head][..., None, None]


PLAIN = {"tables": _plain_tables, "append": _plain_append, "attend": _plain_attend, "bounds": _plain_bounds, "sparse": _plain_sparse}


# -------------------------------------------------------------------------------------- work
def work(case):
    B, bs = case["batch"], case["bs"]
    mean, new = (case["lo"] + case["hi"]) / 2, (case.get("new_lo", 0) + case.get("new_hi", 0)) / 2
    if case["op"] == "tables" and case["what"] == "release":
        return {"bytes": B * 12 + 0.25 * B * 8 * (mean / bs + 0.5), "flops": 0}
    if case["op"] == "tables":
        return {"bytes": B * 16 + B * new * 4 + B * (new / bs) * 8, "flops": 0}
    H, D = case["hkv"], case["d"]
    if case["op"] in ("append", "bounds"):
        eb = {"f16": 2, "bf16": 2, "f32": 4}[case["dtype"]]
        T, blocks = B * new, B * max(1.0, new / bs)
        if case["op"] == "append":
            return {"bytes": 2 * T * H * D * (eb + 1) + 2 * blocks * H * 4 + 4 * T, "flops": 4 * T * H * D}
        return {"bytes": T * H * D * eb + blocks * H * (2 * D + 4) + 4 * T, "flops": 3 * T * H * D}
    kvb = {"f8": 1, "f16": 2, "bf16": 2}[case.get("kv", "f8")]
    blocks, read = B * mean / bs, B * mean
    extra = 0.0
    if case["op"] == "sparse":
        read = min(read, B * case["budget"] * bs)
        extra = blocks * H * (2 * D + 4)
    return {"bytes": 2 * read * H * D * kvb + extra + B * case["hq"] * D * 6, "flops": 4 * read * case["hq"] * D + 2 * extra * case["hq"] / H}


# --------------------------------------------------------------------------- 64-bit definition
def _e4m3(x):
    """float64 values -> the nearest e4m3 values (ties to even), |x| <= 448."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 4).clamp_min(-9).double())     # 4 significant bits; 2^-9 below 2^-6
    return torch.round(x / step) * step


def exact(case, seed):
    """The operators' floating outputs from their definitions, in float64; None where outputs are whole numbers only."""
    if case["op"] in ("tables", "bounds"):
        return None
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return _exact_append(st) if case["op"] == "append" else _exact_attention(st)


def _exact_append(st):
    bs = st["case"]["bs"]
    slots = st["slots"].long().cpu()
    # runs of consecutive slots inside one block, one after another
    ls = slots.tolist()
    cut = [t for t in range(len(ls)) if t == 0 or ls[t] != ls[t - 1] + 1 or ls[t] % bs == 0]
    first = torch.tensor(cut)
    size = torch.diff(torch.cat([first, torch.tensor([slots.numel()])])).cuda()
    run = torch.repeat_interleave(torch.arange(first.numel(), device="cuda"), size)
    block, start = (slots[first] // bs).cuda(), (slots[first] % bs).cuda()
    res = {}
    for what in "kv":
        x = st[what + "_new"].double()
        T, H, D = x.shape
        codes, scales = st[what + "_cache"].double(), st[what + "_scales"].double()
        amax = torch.zeros(first.numel(), H, dtype=torch.float64, device="cuda").index_reduce_(0, run, x.abs().amax(dim=2), "amax")
        need = torch.where(amax > 0, torch.ceil(torch.log2(amax.clamp_min(1e-300) / 448.0) - 1e-13), torch.full_like(amax, -96.0)).clamp_min(-96.0)
        need = torch.where(amax > 448.0 * torch.exp2(need), need + 1, need)
        s_new = torch.exp2(need)
        s_old = scales[block]
        s = torch.where((start == 0)[:, None], s_new, torch.maximum(s_old, s_new))
        held = codes[block]
        again = _e4m3(held * (s_old / s).clamp_max(1.0)[:, :, None, None])
        before = torch.arange(bs, device="cuda")[None, :] < start[:, None]
        codes[block] = torch.where(before[:, None, :, None], again, held)
        at = st["slots"].long()
        codes[at // bs, :, at % bs] = _e4m3(x / s[run][:, :, None])
        scales[block] = s
        res[what], res[what + "s"] = codes, scales
    return res


def _exact_attention(st):
    c = st["case"]
    B, H, D, bs = c["batch"], c["hkv"], c["d"], c["bs"]
    G = c["hq"] // H
    out = torch.zeros(B, c["hq"], D, dtype=torch.float64, device="cuda")

    def rows(what, ids, h):
        x = st[what + "_cache"]
        if st[what + "_scales"] is None:
            return x[ids, h].double()
        return x.view(torch.uint8)[ids, h].view(torch.float8_e4m3fn).double() * st[what + "_scales"][ids, h].double()[:, None, None]

    lens = st["lens"].tolist()
    for b in range(B):
        L = lens[b]
        nblk = -(-L // bs)
        if not nblk:
            continue
        ids = st["block_tables"][b, :nblk].long()
        for h in range(H):
            q = st["q"][b, h * G:(h + 1) * G].double()
            j = torch.arange(nblk, device="cuda")
            if c["op"] == "sparse" and nblk > c["budget"]:
                top = float(q.abs().max())
                e = -96 if top == 0 else max(-96, math.ceil(math.log2(top / 127.0) - 1e-13))
                e += top > 127.0 * 2.0 ** e
                qi = torch.round(q / 2.0 ** e)
                bd = st["bounds"][ids, h].double()
                best = torch.maximum(qi[:, None] * bd[None, :, 0], qi[:, None] * bd[None, :, 1]).sum(dim=2).amax(dim=0)
                score = best * torch.exp2(st["bound_exps"][ids, h].double())
                order = sorted(range(nblk - 1), key=lambda i, s=score.tolist(): (-s[i], i))
                j = torch.tensor(sorted(order[:c["budget"] - 1]) + [nblk - 1], device="cuda")
            k, v = rows("k", ids[j], h).reshape(-1, D), rows("v", ids[j], h).reshape(-1, D)
            n = k.shape[0] - (nblk * bs - L)               # only the newest block can be partly filled
            w = torch.softmax((q @ k[:n].T) * st["scale"], dim=1)
            out[b, h * G:(h + 1) * G] = w @ v[:n]
    return {"out": out, "selected": None} if c["op"] == "sparse" else {"out": out}
