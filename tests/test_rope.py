"""Rotary positions (kv_rope_frequencies, kv_rope_rotate, kv_rope_append) against
float64 references."""
import ctypes
import math

import numpy as np
import pytest
import torch

import block_reference as R
from paged_kv_cache_273_gb300 import pkv

DEV = "cuda"
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
POOL = {"f16": pkv.PKV_F16, "bf16": pkv.PKV_BF16, "f32": pkv.PKV_F32, "f8": pkv.PKV_F8}
SCALINGS = {
    "plain": dict(base=10000.0),
    "linear": dict(base=10000.0, factor=4.0),
    "parts": dict(base=10000.0, factor=16.0, trained_len=4096, low=1.0, high=32.0),
    "wavelength": dict(base=500000.0, factor=8.0, trained_len=8192, low=1.0, high=4.0),
}


def thetas(rot, scaling):
    """Radians a position and the magnitude, float64, one pair after another."""
    c = dict(factor=1.0, trained_len=0, low=0.0, high=0.0)
    c.update(SCALINGS[scaling])
    out = []
    for i in range(rot // 2):
        f = c["base"] ** (-2.0 * i / rot)
        if scaling == "linear":
            f /= c["factor"]
        elif scaling == "parts":
            def at(turns):
                return rot * math.log(c["trained_len"] / (turns * 2 * math.pi)) / (2 * math.log(c["base"]))
            first, last = max(0, math.floor(at(c["high"]))), min(rot - 1, math.ceil(at(c["low"])))
            s = min(1.0, max(0.0, (i - first) / max(last - first, 0.001)))
            f = f / c["factor"] * s + f * (1 - s)
        elif scaling == "wavelength":
            wave = 2 * math.pi / f
            if wave > c["trained_len"] / c["low"]:
                f /= c["factor"]
            elif wave > c["trained_len"] / c["high"]:
                s = (c["trained_len"] / wave - c["low"]) / (c["high"] - c["low"])
                f = (1 - s) * f / c["factor"] + s * f
        out.append(f)
    return np.array(out), 0.1 * math.log(c["factor"]) + 1.0 if scaling == "parts" else 1.0


def turn(x, positions, rot, layout, scaling, back=False):
    """x [T, H, D] float64 -> (rotated, error bound of an fp32 computation).

    The bound: a sine or cosine of CUDA's sincospif is off by at most 2 units in the last
    place (2^-23 below 1), its angle by 2 pi 2^-32, the frequencies' words (a double's 53
    bits of a turn below 0.16) times a position below 2^31 by 2 pi 2^-24 at most, so
    2^-21 here for far positions; the magnitude, the product and the fma round three times,
    2^-24 each.  All relative to m (|a| + |b|): 2^-23 + 2^-29 + 3 * 2^-24 < 2^-21 for
    positions up to 2^24."""
    th, m = thetas(rot, scaling)
    ang = np.asarray(positions, np.float64)[:, None] * th
    c, s = (m * np.cos(ang))[:, None, :], (m * np.sin(ang))[:, None, :] * (-1 if back else 1)
    y, tol = x.copy(), np.zeros_like(x)
    lo = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    a, b = x[..., lo[0]], x[..., lo[1]]
    y[..., lo[0]], y[..., lo[1]] = a * c - b * s, b * c + a * s
    for part in lo:
        tol[..., part] = (np.abs(a) + np.abs(b)) * m * 2.0 ** -21
    return y, tol


def rounded(y, tol, dtype):
    """The bound of y rounded to dtype: half a step, relative, or of the smallest subnormal."""
    eps, tiny = torch.finfo(DT[dtype]).eps, {"f16": 2.0 ** -24, "bf16": 2.0 ** -133, "f32": 2.0 ** -149}[dtype]
    return tol + eps / 2 * (np.abs(y) + tol) + tiny / 2


def close(got, y, tol, dtype):
    err, lim = np.abs(got.double().cpu().numpy() - y), rounded(y, tol, dtype)
    bad = err > lim
    assert not bad.any(), (int(bad.sum()), float((err - lim).max()))


# --------------------------------------------------------------------------- CPU
@pytest.mark.parametrize("scaling", list(SCALINGS))
@pytest.mark.parametrize("rot", [16, 48, 64, 128])
def test_frequencies(rot, scaling):
    words, m = pkv.kv_rope_frequencies(rot, scaling=scaling, **SCALINGS[scaling])
    th, want_m = thetas(rot, scaling)
    assert words.size == rot // 2 and abs(m - want_m) < 1e-6
    got = words.astype(np.float64) / 2.0 ** 64
    # a few roundings of a double
    assert np.all(np.abs(got - th / (2 * math.pi)) <= 1e-15 * th + 2.0 ** -64)


def test_angle_is_the_product_modulo_a_turn():
    # what the kernel multiplies: a word times a position, modulo 2^64
    words, _ = pkv.kv_rope_frequencies(128)
    th, _ = thetas(128, "plain")
    for pos in (0, 1, 4095, 131071, 10 ** 6, -7):
        for i in (0, 1, 17, 63):
            turns = (int(words[i]) * pos) % 2 ** 64 / 2.0 ** 64
            assert abs(math.cos(2 * math.pi * turns) - math.cos(pos * th[i])) < 1e-9


def test_frequency_refusals():
    inv, uns = pkv.PKV_ERR_INVALID, pkv.PKV_ERR_UNSUPPORTED

    def status(**kw):
        args = dict(rot_dim=64, base=10000.0, scaling="plain")
        args.update(kw)
        with pytest.raises(pkv.PkvError) as e:
            pkv.kv_rope_frequencies(**args)
        return e.value.status
    for r in (0, 8, 20, 144, -16):
        assert status(rot_dim=r) == uns
    for b in (0.5, float("inf"), float("nan"), -1.0):
        assert status(base=b) == inv
    for f in (0.0, -1.0, float("nan"), float("inf")):
        assert status(scaling="linear", factor=f) == inv
    for kw in (dict(trained_len=0, low=1.0, high=2.0), dict(trained_len=4096, low=0.0, high=2.0),
               dict(trained_len=4096, low=2.0, high=2.0), dict(trained_len=4096, low=1.0, high=float("nan"))):
        assert status(scaling="parts", factor=2.0, **kw) == inv
        assert status(scaling="wavelength", factor=2.0, **kw) == inv
    assert status(scaling="parts", base=1.0, factor=2.0, trained_len=4096, low=1.0, high=2.0) == inv
    with pytest.raises(ValueError):
        pkv.kv_rope_frequencies(64, scaling="other")
    f, m = (ctypes.c_uint64 * 32)(), ctypes.c_float()
    lib = pkv.load()
    assert lib.kv_rope_frequencies(64, 10000.0, 7, 1.0, 0, 0.0, 0.0, f, ctypes.byref(m)) == inv
    assert lib.kv_rope_frequencies(64, 10000.0, 0, 1.0, 0, 0.0, 0.0, None, ctypes.byref(m)) == inv
    assert lib.kv_rope_frequencies(64, 10000.0, 0, 1.0, 0, 0.0, 0.0, f, None) == inv


def _buffer():
    buf = (ctypes.c_uint8 * 8192)()
    return buf, (ctypes.addressof(buf) + 15) // 16 * 16


def test_rotate_refusals():
    lib = pkv.load()
    keep, a = _buffer()
    inv, uns = pkv.PKV_ERR_INVALID, pkv.PKV_ERR_UNSUPPORTED

    def call(rope=None, x=a, xs=256, dt=pkv.PKV_F16, heads=2, D=128, pos=a, n=1, out=a, os_=256, **kw):
        r = pkv.Rope(kw.get("freqs", a), kw.get("rot", 64), kw.get("layout", 0), kw.get("mag", 1.0))
        return lib.kv_rope_rotate(None if rope == 0 else ctypes.byref(r), x, xs, dt, heads, D, pos, n, 0, out, os_, None)
    assert call(rope=0) == inv and call(freqs=None) == inv and call(freqs=a + 8) == inv
    assert call(layout=2) == inv and call(mag=float("nan")) == inv
    for rot in (0, 8, 72, 144):
        assert call(rot=rot) == uns
    assert call(rot=128, D=64, heads=2, xs=128, os_=128) == uns
    for dt in (pkv.PKV_I8, pkv.PKV_I4, pkv.PKV_F8, 9):
        assert call(dt=dt) == uns
    assert call(D=96) == uns and call(n=-1) == inv and call(heads=-1) == inv and call(heads=70000) == inv
    assert call(x=None) == inv and call(out=None) == inv and call(pos=None) == inv
    assert call(x=a + 8) == inv and call(out=a + 2) == inv and call(pos=a + 2) == inv
    assert call(xs=255) == inv and call(xs=260) == inv and call(os_=128) == inv and call(xs=-256) == inv
    assert call(xs=512) == inv                       # in place, but another stride
    assert call(n=0, x=None) == pkv.PKV_OK and call(heads=0, x=None) == pkv.PKV_OK


def test_append_refusals():
    lib = pkv.load()
    keep, a = _buffer()
    b = a + 4096
    inv, uns = pkv.PKV_ERR_INVALID, pkv.PKV_ERR_UNSUPPORTED
    pools = {k: pkv.kv_block_pool_init(8, 16, 2, 64, t) for k, t in POOL.items()}
    pools["i8"] = pkv.kv_block_pool_init(8, 16, 2, 64, pkv.PKV_I8)

    def call(pool="bf16", rope=None, q=a, qs=256, k=a, ks=128, v=a, vs=128, dt=pkv.PKV_BF16, hq=4, pos=a, slots=a, n=1,
             qo=b, qos=256, kc=a, vc=a, ksc=None, vsc=None, **kw):
        r = pkv.Rope(kw.get("freqs", a), kw.get("rot", 64), 0, 1.0)
        return lib.kv_rope_append(None if pool is None else pools[pool].handle, None if rope == 0 else ctypes.byref(r), q, qs,
                                  k, ks, v, vs, dt, hq, pos, slots, n, qo, qos, kc, vc, ksc, vsc, None)
    assert call(pool=None) == inv and call(rope=0) == inv and call(freqs=None) == inv
    assert call(rot=128) == uns and call(pool="i8", dt=pkv.PKV_F16, ksc=a, vsc=a) == uns
    assert call(dt=pkv.PKV_F16) == inv and call(pool="f8") == inv          # (no scales)
    assert call(pool="f8", dt=pkv.PKV_I8, ksc=a, vsc=a) == uns
    for name in ("k", "v", "pos", "slots", "kc", "vc", "q", "qo"):
        assert call(**{name: None}) == inv, name
        assert call(**{name: a + 2}) == inv, name
    for kw in (dict(ks=120), dict(vs=127), dict(qs=128), dict(qos=252), dict(n=-1), dict(hq=-1), dict(hq=70000), dict(ks=132),
               dict(qo=a, qos=512)):
        assert call(**kw) == inv, kw
    assert call(n=0, k=None) == pkv.PKV_OK
    if not torch.cuda.is_available():
        assert call() == pkv.PKV_ERR_CUDA
        assert call(q=None, qo=None, hq=0) == pkv.PKV_ERR_CUDA


def test_binding_refusals():
    freqs, m = pkv.kv_rope_frequencies(64)
    with pytest.raises(ValueError):
        pkv.RopePlan(freqs, m, "other", device="cpu")
    plan = pkv.RopePlan(freqs, m, "half", device="cpu")
    x, p = torch.zeros(3, 2, 64, dtype=torch.float16), torch.zeros(3, dtype=torch.int32)
    for bad in (x[0], x.to(torch.int8), x):           # (the last: not on a GPU)
        with pytest.raises(ValueError):
            pkv.kv_rope_rotate(plan, bad, p)


# --------------------------------------------------------------------------- GPU
def rows(T, H, D, dtype, seed, pad=0):
    """Rows [T, H, D] inside wider ones (pad heads on either side), and the whole tensor."""
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(T, H + 2 * pad, D, generator=g) * 2).to(DT[dtype]).to(DEV)
    return w[:, pad:pad + H], w


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).to(DEV)


CASES = [  # T, heads, D, rot, layout, scaling, dtype
    (1, 1, 64, 16, "half", "plain", "f16"),
    (1, 40, 128, 128, "half", "wavelength", "bf16"),
    (3, 5, 64, 64, "interleaved", "parts", "f32"),
    (17, 9, 128, 48, "half", "linear", "f32"),
    (33, 12, 64, 32, "interleaved", "plain", "bf16"),
    (300, 7, 128, 96, "interleaved", "parts", "f16"),
    (257, 33, 64, 48, "half", "wavelength", "f16"),
    (5000, 10, 128, 64, "half", "parts", "bf16"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_gpu_rotate(case, back):
    T, H, D, rot, layout, scaling, dtype = case
    x, whole = rows(T, H, D, dtype, 1, pad=1)
    before = whole.clone()
    rng = np.random.default_rng(T)
    pos = rng.integers(0, 2 ** 20, T)
    pos[0] = 0
    plan = pkv.rope_plan(rot, layout=layout, scaling=scaling, **SCALINGS[scaling])
    out = pkv.kv_rope_rotate(plan, x, i32(pos), transposed=back)
    y, tol = turn(x.double().cpu().numpy(), pos, rot, layout, scaling, back)
    close(out, y, tol, dtype)
    assert torch.equal(out[..., rot:], x[..., rot:])          # bit for bit
    # in place, and into rows of another stride: the same values, the neighbours untouched
    wide = torch.full((T, H + 3, D), 7.0, dtype=x.dtype, device=DEV)
    pkv.kv_rope_rotate(plan, x, i32(pos), wide[:, 1:1 + H], transposed=back)
    assert torch.equal(wide[:, 1:1 + H], out) and bool((wide[:, 0] == 7).all()) and bool((wide[:, 1 + H:] == 7).all())
    assert torch.equal(whole, before)
    pkv.kv_rope_rotate(plan, x, i32(pos), x, transposed=back)
    assert torch.equal(x, out) and torch.equal(whole[:, 0], before[:, 0]) and torch.equal(whole[:, -1], before[:, -1])


@pytest.mark.gpu
def test_gpu_rotate_extreme_positions():
    """The whole range of positions: the angles' error is then the frequencies' own, 2 pi 2^-24."""
    pos = np.array([2 ** 31 - 1, -2 ** 31, -1, 1, 2 ** 30 + 12345, 131071, 0])
    x, _ = rows(len(pos), 2, 128, "f32", 3)
    plan = pkv.rope_plan(128)
    out = pkv.kv_rope_rotate(plan, x, i32(pos)).double().cpu().numpy()
    words, _ = pkv.kv_rope_frequencies(128)
    xs = x.double().cpu().numpy()
    for t, p in enumerate(pos):
        # the definition for the words: exact integers
        a = np.array([(int(w) * int(p)) % 2 ** 64 / 2.0 ** 64 * 2 * math.pi for w in words])
        lo, hi = xs[t, :, :64], xs[t, :, 64:]
        want = np.concatenate([lo * np.cos(a) - hi * np.sin(a), hi * np.cos(a) + lo * np.sin(a)], axis=1)
        lim = (np.abs(lo) + np.abs(hi)) * 2.0 ** -21
        assert np.all(np.abs(out[t] - want) <= np.concatenate([lim, lim], axis=1) + np.abs(want) * 2.0 ** -24), p


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gpu_gradient(layout):
    """The transposed rotation is the gradient: against autograd of the formula in float64, and
    against differences (the rotation is linear, so a difference of any size is one)."""
    T, H, D, rot = 19, 3, 64, 48
    plan = pkv.rope_plan(rot, layout=layout, scaling="parts", **SCALINGS["parts"])
    pos = np.arange(T) * 977
    x, _ = rows(T, H, D, "f32", 5)
    g, _ = rows(T, H, D, "f32", 6)
    got = pkv.kv_rope_rotate(plan, g, i32(pos), transposed=True).double().cpu()
    th, m = thetas(rot, "parts")
    xd = x.double().cpu().requires_grad_(True)
    ang = torch.from_numpy(pos[:, None] * th)[:, None, :]
    a, b = (xd[..., :rot // 2], xd[..., rot // 2:rot]) if layout == "half" else (xd[..., 0:rot:2], xd[..., 1:rot:2])
    ya, yb = m * (a * ang.cos() - b * ang.sin()), m * (b * ang.cos() + a * ang.sin())
    ga, gb = (g[..., :rot // 2], g[..., rot // 2:rot]) if layout == "half" else (g[..., 0:rot:2], g[..., 1:rot:2])
    loss = (ya * ga.double().cpu()).sum() + (yb * gb.double().cpu()).sum() + (xd[..., rot:] * g[..., rot:].double().cpu()).sum()
    loss.backward()
    _, tol = turn(g.double().cpu().numpy(), pos, rot, layout, "parts", True)
    close(got, xd.grad.numpy(), tol, "f32")
    d, _ = rows(T, H, D, "f32", 7)
    step = (pkv.kv_rope_rotate(plan, x + d, i32(pos)).double() - pkv.kv_rope_rotate(plan, x, i32(pos)).double()).cpu()
    lhs, rhs = float((step * g.double().cpu()).sum()), float((d.double().cpu() * got).sum())
    # x + d and both rotations round in fp32: 2^-24 relative twice, 2^-21 of |a| + |b| twice
    lim = float((g.double().abs().cpu() * (x.double().abs() + d.double().abs()).cpu().amax()).sum()) * 8 * 2.0 ** -21
    assert abs(lhs - rhs) <= lim


APPENDS = [  # lens, new, hq, hkv, D, bs, rot, layout, scaling, dtype, kv
    ([0], [1], 1, 1, 64, 8, 64, "half", "plain", "f16", "f16"),
    ([5, 0, 131], [1, 1, 1], 8, 2, 128, 16, 128, "half", "wavelength", "bf16", "bf16"),
    ([0, 3, 16, 1], [33, 0, 17, 5], 6, 3, 64, 16, 32, "interleaved", "parts", "f32", "f32"),
    ([7, 100], [60, 9], 0, 2, 128, 4, 48, "half", "linear", "bf16", "bf16"),
    ([0, 9, 31], [1, 1, 1], 4, 2, 64, 32, 64, "half", "plain", "bf16", "f8"),
    ([0, 3, 15, 16, 250], [300, 13, 1, 40, 9], 8, 2, 128, 16, 128, "interleaved", "parts", "f16", "f8"),
    ([0, 5], [500, 290], 4, 1, 64, 256, 48, "half", "wavelength", "f32", "f8"),
    ([1, 2], [77, 3], 0, 3, 128, 64, 64, "interleaved", "linear", "f32", "f8"),
    ([0] * 40, [97] * 40, 4, 4, 128, 16, 128, "half", "plain", "bf16", "f8"),
]


def _append_state(case, seed=0):
    lens, new, hq, H, D, bs, rot, layout, scaling, dtype, kv = case
    rng = np.random.default_rng(seed)
    start = [n % bs for n in lens]
    need = [-(-(s + n) // bs) for s, n in zip(start, new)]
    nb = sum(need) + 5
    ids = rng.permutation(nb)
    slots, pos, at = [], [], 0
    for L, s, n, m in zip(lens, start, new, need):
        for i in range(n):
            slots.append(int(ids[at + (s + i) // bs]) * bs + (s + i) % bs)
            pos.append(L + i)
        at += m
    T = len(slots)
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn(T, hq + 2 * H, D, generator=g) * 2).to(DT[dtype]).to(DEV)
    pool = pkv.kv_block_pool_init(nb, bs, H, D, POOL[kv])
    kc, vc, ks, vs = pool.alloc_cache()
    for c in (kc, vc):
        c.view(torch.uint8).copy_(torch.randint(0, 120, c.view(torch.uint8).shape, generator=g, dtype=torch.uint8))
    for s in (ks, vs):
        if s is not None:
            s.copy_(torch.exp2(torch.randint(-12, -6, s.shape, generator=g).float()))
    plan = pkv.rope_plan(rot, layout=layout, scaling=scaling, **SCALINGS[scaling])
    return dict(pool=pool, plan=plan, q=qkv[:, :hq], k=qkv[:, hq:hq + H], v=qkv[:, hq + H:], slots=slots, pos=pos, kc=kc, vc=vc, ks=ks, vs=vs,
                q_out=torch.full((T, hq, D), 9.0, dtype=DT[dtype], device=DEV))


def _append(s, slots=None, stream=None):
    hq = s["q"].shape[1]
    pkv.kv_rope_append(s["pool"], s["plan"], s["q"] if hq else None, s["k"], s["v"], i32(s["pos"]), i32(s["slots"] if slots is None else slots),
                       s["q_out"] if hq else None, s["kc"], s["vc"], s["ks"], s["vs"], stream=stream)


@pytest.mark.gpu
@pytest.mark.parametrize("case", APPENDS, ids=range(len(APPENDS)))
def test_gpu_append(case):
    lens, new, hq, H, D, bs, rot, layout, scaling, dtype, kv = case
    s = _append_state(case)
    slots, pos = np.array(s["slots"]), np.array(s["pos"])
    was = {n: s[n].clone() if s[n] is not None else None for n in ("kc", "vc", "ks", "vs")}
    _append(s)
    assert pkv.pkv_check_error(s["pool"]) == pkv.PKV_OK
    # q and K are what kv_rope_rotate makes of them, which is right to its bound
    if hq:
        assert torch.equal(s["q_out"], pkv.kv_rope_rotate(s["plan"], s["q"], i32(pos)))
    turned = pkv.kv_rope_rotate(s["plan"], s["k"], i32(pos))
    y, tol = turn(s["k"].double().cpu().numpy(), pos, rot, layout, scaling)
    close(turned, y, tol, dtype)
    if kv != "f8":
        for n, x in (("kc", turned), ("vc", s["v"])):
            want = was[n].clone()
            want[torch.from_numpy(slots // bs), :, torch.from_numpy(slots % bs)] = x
            assert torch.equal(s[n].view(torch.uint8), want.view(torch.uint8)), n
        return
    # 8-bit floats: codes and scales of K's fp32 values, bit for bit, by the reference's append
    k32 = pkv.kv_rope_rotate(s["plan"], s["k"].float(), i32(pos)).double().cpu().numpy()
    for n, m, x in (("kc", "ks", k32), ("vc", "vs", s["v"].double().cpu().numpy())):
        codes, scales = was[n].view(torch.uint8).cpu().numpy().copy(), was[m].double().cpu().numpy().copy()
        R.append_f8(x, slots, bs, codes, scales)
        assert np.array_equal(s[m].double().cpu().numpy(), scales), m
        got = s[n].view(torch.uint8).cpu().numpy()
        assert np.array_equal(R.E4M3[got], R.E4M3[codes]), n


@pytest.mark.gpu
@pytest.mark.parametrize("case", [APPENDS[1], APPENDS[5]], ids=["bf16", "f8"])
def test_gpu_append_padding_and_bad_slots(case):
    s = _append_state(case, 3)
    good = _append_state(case, 3)
    T, bs = len(s["slots"]), case[5]
    total = s["pool"].num_blocks * bs
    # (none inside a block: a block gets at most one run of new rows a call)
    skip = {0: -1, T - 1: total, min(T // 2, 175): 2 ** 31 - 1}
    slots = [skip.get(t, x) for t, x in enumerate(s["slots"])]
    _append(s, slots)
    assert pkv.pkv_check_error(s["pool"]) == pkv.PKV_ERR_BAD_INDEX
    assert pkv.pkv_check_error(s["pool"]) == pkv.PKV_OK
    for t in skip:
        assert bool((s["q_out"][t] == 9).all())
    # the others as in a call without the skipped tokens
    live = [t for t in range(T) if t not in skip]
    sub = dict(good, q=good["q"][live], k=good["k"][live], v=good["v"][live], pos=[good["pos"][t] for t in live], q_out=good["q_out"][live].contiguous())
    _append(sub, [good["slots"][t] for t in live])
    assert torch.equal(s["q_out"][live], sub["q_out"])
    for n in ("kc", "vc", "ks", "vs"):
        if s[n] is not None:
            assert torch.equal(s[n].view(torch.uint8), sub[n].view(torch.uint8)), n


@pytest.mark.gpu
def test_gpu_append_in_place_stream_and_graph():
    """q rotated in place, on a side stream; then captured and replayed on other inputs."""
    case = APPENDS[5]
    ref, s = _append_state(case, 4), _append_state(case, 4)
    _append(ref)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    q = s["q"]
    pos, slots = i32(s["pos"]), i32(s["slots"])
    torch.cuda.synchronize()
    keep = {n: s[n].clone() for n in ("kc", "vc", "ks", "vs")}
    q_before = q.clone()
    pkv.kv_rope_append(s["pool"], s["plan"], q, s["k"], s["v"], pos, slots, q, s["kc"], s["vc"], s["ks"], s["vs"], stream=stream)
    stream.synchronize()
    assert torch.equal(q, ref["q_out"])
    for n in keep:
        assert torch.equal(s[n].view(torch.uint8), ref[n].view(torch.uint8)), n
    q.copy_(q_before)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.kv_rope_append(s["pool"], s["plan"], q, s["k"], s["v"], pos, slots, s["q_out"], s["kc"], s["vc"], s["ks"], s["vs"])
    for n in keep:
        s[n].copy_(keep[n])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(s["q_out"], ref["q_out"])
    for n in keep:
        assert torch.equal(s[n].view(torch.uint8), ref[n].view(torch.uint8)), n


@pytest.mark.gpu
def test_gpu_empty_calls():
    plan = pkv.rope_plan(64)
    x = torch.zeros(0, 4, 64, dtype=torch.float16, device=DEV)
    assert pkv.kv_rope_rotate(plan, x, i32([])).shape == (0, 4, 64)
    s = _append_state(([0], [0], 2, 1, 64, 16, 64, "half", "plain", "f16", "f16"))
    _append(s)
    assert pkv.pkv_check_error(s["pool"]) == pkv.PKV_OK
    with pytest.raises(ValueError):
        pkv.kv_rope_rotate(plan, torch.zeros(2, 64, 4, dtype=torch.float16, device=DEV).transpose(1, 2), i32([0, 1]))


@pytest.mark.gpu
def test_gpu_rotate_on_a_stream_of_its_own():
    """Into a given tensor; a new one would be the current stream's."""
    plan = pkv.rope_plan(64)
    x = torch.randn(500, 4, 64, device=DEV)
    pos = i32(list(range(500)))
    want = pkv.kv_rope_rotate(plan, x, pos)
    out, stream = torch.zeros_like(x), torch.cuda.Stream()
    torch.cuda.synchronize()
    with pytest.raises(ValueError):
        pkv.kv_rope_rotate(plan, x, pos, stream=stream)
    assert pkv.kv_rope_rotate(plan, x, pos, out, stream=stream) is out
    stream.synchronize()
    assert torch.equal(out, want)
    with torch.cuda.stream(stream):                    # the current stream: a new tensor is its own
        assert torch.equal(pkv.kv_rope_rotate(plan, x, pos), want)
    stream.synchronize()
