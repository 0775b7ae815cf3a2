"""Recurrent-state cache (cache_store / cache_load / cache_step) against a plain fp64 evaluation.

Tolerances, with u = 2^-24. Storing: scale and the product with its reciprocal are off by at most 4 u together, so
a stored value differs from the true one by at most half a code step (int8: scale / 2; e4m3: 2^-4 of the value, or
2^-10 scale below its normal range) plus 6 u |S|. Reading: the window's exponents are sums of up to W log decays,
each sum off by W u |D|, the exponential by 4 u; an entry is a sum of W + 1 products, off by (W + 4) u of the sum
of their magnitudes. A step's output sums Dk + W such terms in any order: (Dk + 2 W + 16) u of the sum of the
magnitudes, plus eps / 2 of its type.
"""
import ctypes

import numpy as np
import pytest
import torch

import chunkwise_linear_rnn_gla_b200 as gla
from chunkwise_linear_rnn_gla_b200 import _lib, build as gbuild, cache as gc, scan

U = 2.0 ** -24
TAU = 16.0


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return _lib.load()


def scales64(c, at=slice(None)):
    """scale [slots,H,Dk,groups] spread over the columns, fp64"""
    return np.repeat(c.scale[at].double().cpu().numpy(), 128, -1)[..., : c.Dv]


def codes64(c, at=slice(None)):
    return c.codes.view(torch.uint8)[at].view(c.codes.dtype).float().double().cpu().numpy()


def stored64(c, at=slice(None)):
    return codes64(c, at) * scales64(c, at)


def half_code(S, scale, fmt):
    """Half a step of the code that holds S (fp64 values and their scales)."""
    return 0.5 * scale if fmt == "int8" else np.maximum(np.abs(S) * 2.0 ** -4, scale * 2.0 ** -10)


def group_max(S):
    V = S.shape[-1]
    G = -(-V // 128)
    return np.stack([np.abs(S[..., 128 * i:128 * (i + 1)]).max(-1) for i in range(G)], -1)


def check_stored(c, at, S, eS):
    """The pool's slots `at` hold S (fp64, computed in fp32 within eS)."""
    lim = 127.0 if c.format == "int8" else 448.0
    want = group_max(S) / lim
    tol = group_max(eS) / lim * (np.ones_like(want)) + 4 * U * want + 1e-36
    assert (np.abs(c.scale[at].double().cpu().numpy() - want) <= tol).all()
    sc = scales64(c, at)
    got = stored64(c, at)
    assert (np.abs(got - S) <= half_code(np.abs(S) + eS, sc, c.format) + eS + 8 * U * np.abs(S) + 1e-36).all()


def fill_pool(P, H, K, V, W, fmt, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    c = gc.StateCache.empty(P, H, K, V, window=W, format=fmt, dtype=dtype)
    S = r(P, H, K, V) * (0.05 + torch.rand(P, H, K, 1, generator=g))
    gc.cache_store(c, S.cuda(), torch.arange(P, dtype=torch.int32, device="cuda"))
    c.k.copy_((r(P, H, W, K) / K ** 0.5).to(dtype))
    c.v.copy_(r(P, H, W, V).to(dtype))
    c.log_a.copy_(torch.nn.functional.logsigmoid(r(P, H, W, K)) / TAU)
    return c, S, g


def token(c, B, g, gate="channel"):
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    H, K, V = c.H, c.Dk, c.Dv
    z = r(*gla.gate_shape(gate, B, H, None, K))
    return dict(q=(r(B, H, K) / K ** 0.5).to(c.dtype), k=(r(B, H, K) / K ** 0.5).to(c.dtype), v=r(B, H, V).to(c.dtype),
                log_a=z if gate == "preact" else torch.nn.functional.logsigmoid(z) / TAU)


def log_alpha64(z, gate, B, H, K):
    z = z.double().numpy()
    if gate == "preact":
        return (np.minimum(z, 0) - np.log1p(np.exp(-np.abs(z)))) / TAU
    if gate == "scalar":
        return np.broadcast_to(z[..., None], (B, H, K))
    if gate == "head":
        return np.broadcast_to(z[None, :, None], (B, H, K))
    return z


def windowed64(c, base, slot, n, tok=None, b=None, la=None):
    """(state, error bound, sum of magnitudes) of a slot after n window tokens and, with tok, row b of the call."""
    kw, vw, gw = (x[slot].double().cpu().numpy() for x in (c.k, c.v, c.log_a))
    k, v, g = list(kw[:, :n].swapaxes(0, 1)), list(vw[:, :n].swapaxes(0, 1)), list(gw[:, :n].swapaxes(0, 1))
    if tok is not None:
        k.append(tok["k"][b].double().numpy())
        v.append(tok["v"][b].double().numpy())
        g.append(la[b])
    W = c.window
    S, m = base[slot].copy(), np.abs(base[slot])
    D = np.zeros(S.shape[:2])
    for i in range(len(k)):
        e = np.exp(np.maximum(g[i], -1e4))[..., None]
        p = k[i][..., None] * v[i][:, None, :]
        S, m = e * S + p, e * m + np.abs(p)
        D = D + np.abs(np.maximum(g[i], -100.0))
    # a pre-activation gate adds its own error (as for the scan): under 40 u of log a at |z| <= 6
    return S, ((W + 12) * U + (W + 40) * U * D[..., None]) * m, m


def pool_case(c, slots, lengths):
    s = torch.tensor(slots, dtype=torch.int32, device="cuda")
    return s, torch.tensor(lengths, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- store and load

DIMS = [(1, 1, 1), (2, 3, 5), (1, 64, 128), (2, 40, 129), (1, 128, 256), (1, 33, 100), (1, 256, 512), (3, 16, 260)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("H,K,V", DIMS)
def test_store_and_load(lib, H, K, V, fmt):
    P, B = 7, 4
    c, _, g = fill_pool(P, H, K, V, 4, fmt, torch.float32)
    before = [x.clone() for x in (c.codes.view(torch.uint8), c.scale, c.k, c.v, c.log_a)]
    S = torch.randn(B, H, K, V, generator=g) * torch.logspace(-6, 6, K)[None, None, :, None]
    slots, lengths = pool_case(c, [5, -1, 0, 3], [0, 0, 0, 0])
    gc.cache_store(c, S.cuda(), slots)
    assert gla.gla_check_device_error() == _lib.GLA_OK
    live = [0, 2, 3]
    S64 = S.double().numpy()
    check_stored(c, [5, 0, 3], S64[live], 2 * U * np.abs(S64[live]))
    rest = [1, 2, 4, 6]
    for x, y in zip(before, (c.codes.view(torch.uint8), c.scale, c.k, c.v, c.log_a)):
        assert torch.equal(x[rest], y[rest])
    # read back: exactly code times scale; a slot may be named twice, a padding row is zero
    slots2, _ = pool_case(c, [3, 3, -1, 0, 6], [0] * 5)
    out = gc.cache_load(c, slots2).double().cpu().numpy()
    want = stored64(c)
    for i, s in enumerate([3, 3, None, 0, 6]):
        assert np.array_equal(out[i], 0 * out[i] if s is None else want[s].astype(np.float32).astype(np.float64))
    # storing what was read gives the same codes wherever the largest code is the full one
    gc.cache_store(c, torch.from_numpy(out[3:4]).float().cuda(), slots2[4:5])
    a, b = stored64(c)[0], stored64(c)[6]
    assert (np.abs(a - b) <= half_code(a, scales64(c)[0], fmt) + 8 * U * np.abs(a)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_store_special_values(lib, fmt):
    K, V = 6, 300
    c = gc.StateCache.empty(1, 1, K, V, format=fmt)
    S = torch.randn(1, 1, K, V)
    S[0, 0, 0] = 0
    S[0, 0, 1] *= 1e-32
    S[0, 0, 2, 130] = float("inf")
    S[0, 0, 3, 7] = float("nan")
    S[0, 0, 4] *= 1e30
    S[0, 0, 5, :] = torch.arange(V) % 2 * 2.0 - 1
    slot = torch.zeros(1, dtype=torch.int32, device="cuda")
    gc.cache_store(c, S.cuda(), slot)
    out = gc.cache_load(c, slot).cpu()[0, 0]
    assert bool((out[0] == 0).all()) and bool((out[1] == 0).all())
    assert bool(torch.isnan(out[2, 128:256]).all()) and bool(torch.isfinite(out[2, :128]).all())
    assert bool(torch.isnan(out[3, :128]).all()) and bool(torch.isfinite(out[3, 128:]).all())
    S64 = S.double().numpy()[0, 0]
    sc = scales64(c)[0, 0]
    for r in (4, 5):
        assert (np.abs(out[r].double().numpy() - S64[r]) <= half_code(S64[r], sc[r], fmt) + 8 * U * np.abs(S64[r])).all()
    # a non-finite group stays non-finite through a step and does not reach the others
    q = torch.ones(1, 1, K, dtype=torch.bfloat16, device="cuda")
    v = torch.ones(1, 1, V, dtype=torch.bfloat16, device="cuda")
    o = gc.cache_step(c, q, q, v, torch.zeros(1, 1, K, device="cuda"), slot, torch.zeros_like(slot))[0, 0]
    assert bool(torch.isnan(o[:256]).all()) and bool(torch.isfinite(o[256:]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,fmt,W", [(torch.float32, "int8", 1), (torch.bfloat16, "int8", 16),
                                         (torch.bfloat16, "e4m3", 5), (torch.float32, "e4m3", 64)])
@pytest.mark.parametrize("H,K,V", [(2, 3, 5), (1, 64, 128), (2, 40, 260), (1, 128, 256)])
def test_load_in_the_window(lib, H, K, V, dtype, fmt, W):
    P = 9
    c, _, _ = fill_pool(P, H, K, V, W, fmt, dtype, seed=W)
    sl, ln = [8, 2, -1, 2, 0, 5], [0, W - 1, 3, W // 2, 7 * W + W // 3, 2**31 - 1]
    slots, lengths = pool_case(c, sl, ln)
    out = gc.cache_load(c, slots, lengths).double().cpu().numpy()
    base = stored64(c)
    for i, s in enumerate(sl):
        if s < 0:
            assert (out[i] == 0).all()
            continue
        S, e, _ = windowed64(c, base, s, ln[i] % W)
        assert (np.abs(out[i] - S) <= e + 1e-36).all(), i
    assert gla.gla_check_device_error() == _lib.GLA_OK


# ---------------------------------------------------------------- step


def check_step(c, sl, ln, gate, g, seed_note=""):
    B, W, H, K = len(sl), c.window, c.H, c.Dk
    t = token(c, B, g, gate)
    la = log_alpha64(t["log_a"], gate, B, H, K)
    base = stored64(c)
    old = {n: getattr(c, n).clone() for n in ("k", "v", "log_a", "scale")}
    old_codes = c.codes.view(torch.uint8).clone()
    want = {b: windowed64(c, base, s, ln[b] % W, t, b, la) for b, s in enumerate(sl) if s >= 0}
    slots, lengths = pool_case(c, sl, ln)
    d = {n: x.cuda() for n, x in t.items()}
    o = gc.cache_step(c, d["q"], d["k"], d["v"], d["log_a"], slots, lengths, gate=gate,
                      tau=TAU if gate == "preact" else 0.0).double().cpu().numpy()
    assert gla.gla_check_device_error() == _lib.GLA_OK
    eps = torch.finfo(c.dtype).eps / 2
    folded = []
    for b, s in enumerate(sl):
        if s < 0:
            assert (o[b] == 0).all()
            continue
        S, e, m = want[b]
        q = t["q"][b].double().numpy()
        y = (q[..., None] * S).sum(1)
        tol = (np.abs(q)[..., None] * (e + (K + 2 * W + 16) * U * m)).sum(1)
        assert (np.abs(o[b] - y) <= tol + eps * (np.abs(y) + tol) + 1e-36).all(), (b, np.abs(o[b] - y).max(), tol.max())
        n = ln[b] % W
        old["k"][s, :, n], old["v"][s, :, n] = d["k"][b], d["v"][b]
        got = c.log_a[s, :, n].double().cpu().numpy()
        assert (np.abs(got - la[b]) <= 40 * U * np.abs(la[b])).all()
        old["log_a"][s, :, n] = c.log_a[s, :, n]
        if n == W - 1:
            folded.append(s)
            check_stored(c, [s], S[None], e[None])
    for n in ("k", "v", "log_a"):  # nothing else of the windows changed
        assert torch.equal(getattr(c, n), old[n]), n
    rest = [s for s in range(c.slots) if s not in folded]
    assert torch.equal(c.scale[rest], old["scale"][rest])
    assert torch.equal(c.codes.view(torch.uint8)[rest], old_codes[rest])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,fmt,W", [(torch.float32, "int8", 1), (torch.bfloat16, "int8", 16),
                                         (torch.bfloat16, "e4m3", 5), (torch.float32, "e4m3", 64)])
@pytest.mark.parametrize("H,K,V", [(2, 3, 5), (1, 1, 1), (1, 64, 128), (2, 40, 260), (2, 128, 256), (1, 250, 144)])
def test_step(lib, H, K, V, dtype, fmt, W):
    c, _, g = fill_pool(9, H, K, V, W, fmt, dtype, seed=W + K)
    check_step(c, [8, 2, -1, 7, 0, 5], [0, W - 1, 3, W // 2, 7 * W + W // 3, 2**31 - 1], "channel", g)


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["scalar", "head", "preact"])
def test_step_gate_kinds(lib, gate):
    c, _, g = fill_pool(5, 2, 48, 160, 8, "int8", torch.bfloat16)
    check_step(c, [4, 1, 0], [7, 15, 2], gate, g)


@pytest.mark.gpu
@pytest.mark.parametrize("H,K,V,W", [(4, 256, 512, 16), (2, 512, 128, 16), (1, 320, 64, 32), (1, 64, 1024, 16)])
def test_step_wide(lib, H, K, V, W):
    c, _, g = fill_pool(4, H, K, V, W, "e4m3", torch.bfloat16, seed=1)
    check_step(c, [2, 0, 3], [W - 1, 3, 2 * W + 1], "channel", g)


def many_rows(B, P, W, g, folds):
    """Slots and lengths of a serving batch: every place of the window, some padding rows, `folds` of the rows full."""
    sl = torch.randperm(P, generator=g)[:B].tolist()
    ln = torch.randint(0, 3 * W, (B,), generator=g).tolist()
    for i in range(B):
        if i % 11 == 5:
            sl[i] = -1 - i
        if folds == "none" and ln[i] % W == W - 1 and W > 1:
            ln[i] += 1
        if folds == "all":
            ln[i] = ln[i] // W * W + W - 1
    return sl, ln


@pytest.mark.gpu
@pytest.mark.parametrize("folds", ["some", "none", "all"])
@pytest.mark.parametrize("dtype,fmt,W", [(torch.bfloat16, "int8", 16), (torch.float32, "e4m3", 5)])
@pytest.mark.parametrize("B,H,K,V", [(80, 2, 64, 128), (40, 4, 24, 384), (151, 1, 40, 64), (300, 1, 8, 112),
                                     (38, 4, 128, 256), (75, 2, 520, 16)])
def test_step_many_heads(lib, B, H, K, V, dtype, fmt, W, folds):
    c, _, g = fill_pool(B + 3, H, K, V, W, fmt, dtype, seed=B)
    check_step(c, *many_rows(B, B + 3, W, g, folds), "channel", g)


@pytest.mark.gpu
@pytest.mark.parametrize("gate,W", [("scalar", 8), ("head", 1), ("preact", 2)])
def test_step_many_heads_gate_kinds(lib, gate, W):
    c, _, g = fill_pool(90, 2, 48, 128, W, "int8", torch.bfloat16)
    check_step(c, *many_rows(85, 90, W, g, "some"), gate, g)


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,K,V,W,dtype,fmt,folds", [
    (40, 4, 256, 512, 16, torch.bfloat16, "int8", "some"), (40, 4, 256, 512, 16, torch.bfloat16, "e4m3", "all"),
    (37, 4, 256, 512, 32, torch.bfloat16, "e4m3", "none"), (150, 1, 264, 384, 5, torch.float32, "int8", "some"),
    (76, 2, 104, 1024, 16, torch.bfloat16, "e4m3", "some"), (152, 1, 768, 128, 1, torch.bfloat16, "int8", "some"),
    (149, 1, 56, 1792, 7, torch.bfloat16, "int8", "some"), (148, 1, 256, 512, 3, torch.float32, "e4m3", "all")])
def test_step_many_large_heads(lib, B, H, K, V, W, dtype, fmt, folds):
    c, _, g = fill_pool(B + 2, H, K, V, W, fmt, dtype, seed=1)
    check_step(c, *many_rows(B, B + 2, W, g, folds), "channel" if K != 768 else "preact", g)


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["scalar", "head"])
def test_step_many_large_heads_gate_kinds(lib, gate):
    c, _, g = fill_pool(80, 2, 256, 384, 4, "int8", torch.bfloat16)
    check_step(c, *many_rows(76, 80, 4, g, "some"), gate, g)


@pytest.mark.gpu
def test_step_many_large_heads_refuse_bad_rows(lib):
    """Padding, slots and lengths out of range and slots named twice, folding rows among them: the good rows' results
    are those of a call without the bad ones, to the bit, and nothing else is touched."""
    B, H, K, V, W = 44, 4, 256, 384, 4
    c, _, g = fill_pool(B, H, K, V, W, "e4m3", torch.bfloat16)
    ref, _, _ = fill_pool(B, H, K, V, W, "e4m3", torch.bfloat16)
    sl = torch.randperm(B, generator=g).to(torch.int32)
    ln = torch.randint(0, 3 * W, (B,), generator=g).to(torch.int32)
    good = torch.ones(B, dtype=torch.bool)
    ln[9], ln[30] = W - 1, 2 * W - 1  # both fold, both on row 3's and row 9's slots
    for i, s in ((9, sl[3]), (30, sl[9]), (20, -5), (21, B), (22, 2**31 - 1)):
        sl[i] = s
        good[i] = False
    ln[40], good[40] = -3, False
    t = {n: x.cuda() for n, x in token(c, B, g).items()}
    o = gc.cache_step(c, t["q"], t["k"], t["v"], t["log_a"], sl.cuda(), ln.cuda())
    assert gla.gla_check_device_error() == _lib.GLA_ERR_INVALID_ARG
    pad = torch.where(good, sl, torch.full_like(sl, -1))
    want = gc.cache_step(ref, t["q"], t["k"], t["v"], t["log_a"], pad.cuda(), ln.cuda())
    assert gla.gla_check_device_error() == _lib.GLA_OK
    assert torch.equal(o, want) and bool((o[~good.cuda()] == 0).all())
    for n in ("codes", "scale", "k", "v", "log_a"):
        assert torch.equal(getattr(c, n).view(torch.uint8), getattr(ref, n).view(torch.uint8)), n


@pytest.mark.gpu
def test_step_more_rows_than_a_launch_takes(lib):
    """Over 1024 rows of large heads: a slot that a row of an earlier launch names is refused like any other."""
    B, P, H, K, V, W = 1100, 1060, 1, 768, 128, 2
    c, _, g = fill_pool(P, H, K, V, W, "int8", torch.bfloat16)
    ref, _, _ = fill_pool(P, H, K, V, W, "int8", torch.bfloat16)
    sl = torch.cat([torch.randperm(P, generator=g), torch.full((B - P,), -1)])[torch.randperm(B, generator=g)].to(torch.int32)
    ln = torch.randint(0, 40, (B,), generator=g).to(torch.int32)
    good = sl >= 0
    for i, j in ((1090, 3), (1024, 1023), (700, 699)):
        sl[j], sl[i] = (sl[j] if sl[j] >= 0 else sl[good.nonzero()[0, 0]]), 0
        sl[i] = sl[j]
    # of the rows that name a slot, the first one stands
    seen, good = set(), torch.zeros(B, dtype=torch.bool)
    for i, s in enumerate(sl.tolist()):
        good[i] = s >= 0 and s not in seen
        seen.add(s)
    t = {n: x.cuda() for n, x in token(c, B, g).items()}
    o = gc.cache_step(c, t["q"], t["k"], t["v"], t["log_a"], sl.cuda(), ln.cuda())
    assert gla.gla_check_device_error() == _lib.GLA_ERR_INVALID_ARG
    idx = good.nonzero()[:, 0]
    want = []
    for part in idx.split(100):  # few rows a call: the other kernel
        p = part.cuda()
        want.append(gc.cache_step(ref, *[t[n][p].contiguous() for n in ("q", "k", "v", "log_a")], sl[part].cuda(),
                                  ln[part].cuda()))
    assert gla.gla_check_device_error() == _lib.GLA_OK
    assert bool((o[~good.cuda()] == 0).all())
    # the two kernels sum in different orders: (Dk + 2 W + 16) u of the magnitudes sum |q| |S| (below 2^9 here: |q| sums
    # to under 30, |S| stays under 2^4), and each rounds to bf16
    a, b = o[idx.cuda()].float(), torch.cat(want).float()
    assert float(((a - b).abs() - 2.0 ** -7 * b.abs()).max()) <= 2 * (K + 2 * W + 16) * U * 512
    for n in ("k", "v", "log_a"):
        assert torch.equal(getattr(c, n), getattr(ref, n)), n
    assert float((c.scale / ref.scale.clamp(min=1e-30) - 1).abs().max()) <= 64 * U
    assert int((c.codes.int() - ref.codes.int()).abs().max()) <= 1


@pytest.mark.gpu
def test_step_zero_gates(lib):
    """A zero gate in the window, and one in the call, hide everything before them and nothing after."""
    c, _, g = fill_pool(3, 1, 64, 128, 8, "int8", torch.float32)
    c.log_a[:, :, 3] = -1e30
    c.log_a[:, :, 1, ::2] = 0.0
    check_step(c, [0, 1, 2], [7, 5, 2], "channel", g)
    t = {n: x.cuda() for n, x in token(c, 1, g).items()}
    t["log_a"].fill_(-1e30)
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = gc.cache_step(c, t["q"], t["k"], t["v"], t["log_a"], one, one + 2)
    w = (t["q"] * t["k"]).sum(-1, keepdim=True) * t["v"]
    assert torch.allclose(o, w, rtol=0, atol=float(64 * U * (t["q"] * t["k"]).abs().sum() * t["v"].abs().max()))


@pytest.mark.gpu
def test_step_refuses_bad_rows(lib):
    """Slots and lengths are bounds-checked in the kernel: a bad row is skipped and reported."""
    K, V = 32, 160
    for sl, ln in (([0, 1, 4, 2], [0] * 4), ([0, 1, 2**31 - 1, 2], [0] * 4), ([0, 1, 0, 2], [3] * 4),
                   ([0, 1, 3, 2], [0, 0, -1, 0])):
        c, _, g = fill_pool(4, 2, K, V, 4, "int8", torch.float32)
        ref, _, _ = fill_pool(4, 2, K, V, 4, "int8", torch.float32)
        t = {n: x.cuda() for n, x in token(c, 4, g).items()}
        slots, lengths = pool_case(c, sl, ln)
        o = gc.cache_step(c, t["q"], t["k"], t["v"], t["log_a"], slots, lengths)
        assert gla.gla_check_device_error() == _lib.GLA_ERR_INVALID_ARG
        assert gla.gla_check_device_error() == _lib.GLA_OK
        good = [0, 1, 3]
        pick = {n: x[good].contiguous() for n, x in t.items()}
        want = gc.cache_step(ref, pick["q"], pick["k"], pick["v"], pick["log_a"], slots[good], lengths[good])
        assert torch.equal(o[good], want) and bool((o[2] == 0).all())
        for n in ("codes", "scale", "k", "v", "log_a"):
            assert torch.equal(getattr(c, n).view(torch.uint8), getattr(ref, n).view(torch.uint8)), n
    c, S, g = fill_pool(4, 2, K, V, 4, "e4m3", torch.float32)
    ref, _, _ = fill_pool(4, 2, K, V, 4, "e4m3", torch.float32)
    new = torch.randn(3, 2, K, V, device="cuda")
    for sl in ([1, 1, 3], [1, 4, 3], [1, -2**31, 3]):
        gc.cache_store(c, new, pool_case(c, sl, sl)[0])
        assert gla.gla_check_device_error() == (_lib.GLA_OK if sl[1] < 0 else _lib.GLA_ERR_INVALID_ARG)
        gc.cache_store(ref, new[[0, 2]].contiguous(), pool_case(c, [1, 3], [0, 0])[0])
        assert torch.equal(c.codes.view(torch.uint8), ref.codes.view(torch.uint8)) and torch.equal(c.scale, ref.scale)
    out = gc.cache_load(c, *pool_case(c, [1, 4, 3, 2], [0, 0, -4, 0]))
    assert gla.gla_check_device_error() == _lib.GLA_ERR_INVALID_ARG
    assert bool((out[1] == 0).all()) and bool((out[2] == 0).all()) and bool((out[0] != 0).any())


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,K,V", [(5, 2, 32, 160), (40, 4, 256, 384)])
def test_step_refuses_a_slot_that_a_refused_row_names(lib, B, H, K, V):
    """Both forms of the step: a row whose length is bad is refused, and so is a later row with its slot."""
    c, _, g = fill_pool(B, H, K, V, 4, "int8", torch.bfloat16)
    before = c.codes.clone()
    t = {n: x.cuda() for n, x in token(c, B, g).items()}
    sl = list(range(B))
    sl[3] = 1
    ln = [0] * B
    ln[1] = -1
    o = gc.cache_step(c, t["q"], t["k"], t["v"], t["log_a"], *pool_case(c, sl, ln))
    assert gla.gla_check_device_error() == _lib.GLA_ERR_INVALID_ARG
    assert bool((o[[1, 3]] == 0).all()) and bool((o[[0, 2, 4]] != 0).any(-1).all())
    assert torch.equal(c.codes, before)


@pytest.mark.gpu
def test_cache_on_another_stream_and_in_a_graph(lib):
    """A captured step reads lengths and slots from the device, so a replay advances with them."""
    mk = lambda: fill_pool(6, 2, 64, 128, 4, "int8", torch.bfloat16, seed=8)  # noqa: E731
    (c1, _, g), (c2, _, _) = mk(), mk()
    toks = [{n: x.cuda() for n, x in token(c1, 3, g).items()} for _ in range(6)]
    slots, lengths = pool_case(c1, [5, 0, 2], [0, 3, 1])
    eager, l1 = [], lengths.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for t in toks:
            eager.append(gc.cache_step(c1, t["q"], t["k"], t["v"], t["log_a"], slots, l1))
            l1 += 1
    torch.cuda.synchronize()
    st = {n: x.clone() for n, x in toks[0].items()}
    l2 = lengths.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = gc.cache_step(c2, st["q"], st["k"], st["v"], st["log_a"], slots, l2)
        l2 += 1
    for t, want in zip(toks, eager):
        for n in st:
            st[n].copy_(t[n])
        graph.replay()
        assert torch.equal(o, want)
    for n in ("codes", "scale", "k", "v", "log_a"):
        assert torch.equal(getattr(c1, n).view(torch.uint8), getattr(c2, n).view(torch.uint8)), n


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,limit", [("int8", 0.02), ("e4m3", 0.08)])
def test_prefill_decode_suspend_resume(lib, fmt, limit):
    """The operators together, as a server uses them: two layers (an elementwise recurrence feeding a GLA layer),
    prefill of packed prompts and of a dense batch, states into the pool, decode through slots, a suspended
    sequence resumed as the h0 of another prefill. The fp32 state that gla_step carries is the reference.

    The state is rounded once at the store and once in W = 8 tokens after it. One rounding is off by at most half
    a code, as a root mean square over a row that is normal to within a factor 2 at most
    max / 127 / sqrt(12) < 4.5 / 440 = 1.1% of the row (int8, largest of 128 entries under 4.5 deviations), or
    2^-4 / sqrt(3) = 3.7% (e4m3). The row loses e^G < 0.8 of its old error in W tokens (mean log decay -0.05 a
    token) and takes in one new rounding, so the errors of independent roundings add up to under
    1 / sqrt(1 - 0.64) = 1.7 times one of them. The outputs read the state linearly; the bf16 rounding adds
    0.2%. So 0.02 and 0.08 hold as relative 2-norms over all outputs."""
    B, H, K, V, L, T = 4, 2, 64, 128, 96, 40
    D = H * V
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    bf = torch.bfloat16
    cu = torch.arange(0, (B + 1) * L, L, dtype=torch.int32, device="cuda")
    x = r(1, 1, B * L + T * B, D).to(bf)
    z = r(1, 1, B * L + T * B, D)
    rows = lambda t: t[:, :, B * L:].reshape(T, B, 1, D)  # noqa: E731
    h, hT = scan.scan_fwd(x[:, :, :B * L].contiguous(), z[:, :, :B * L].contiguous(), cu_seqlens=cu, write="leak",
                          gate="preact", tau=TAU)
    pool = torch.zeros(7, 1, D, device="cuda")
    slots = torch.tensor([6, 1, 4, 0], dtype=torch.int32, device="cuda")
    pool[slots.long()] = hT
    v = h.view(B, L, H, V).transpose(1, 2).contiguous()
    q, k = (r(B, H, L + T, K) / K ** 0.5).to(bf), (r(B, H, L + T, K) / K ** 0.5).to(bf)
    la = torch.nn.functional.logsigmoid(r(B, H, L + T, K)) / TAU
    part = lambda t, a, b: t[:, :, a:b].contiguous()  # noqa: E731
    _, S = gla.gla_fwd(part(q, 0, L), part(k, 0, L), v, part(la, 0, L))
    c = gc.StateCache.empty(7, H, K, V, window=8, format=fmt)
    gc.cache_store(c, S, slots)
    lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
    got, want, vs = [], [], []
    for i in range(T):
        hv = scan.scan_step(rows(x)[i], rows(z)[i], pool, slots, write="leak", gate="preact", tau=TAU)
        vi = hv.view(B, H, V)
        vs.append(vi)
        tk = [t[:, :, L + i].contiguous() for t in (q, k)] + [vi, la[:, :, L + i].contiguous()]
        got.append(gc.cache_step(c, *tk, slots, lengths))
        lengths += 1
        want.append(gla.gla_step(*tk, S))
    rel = lambda a, b: float((a.double() - b.double()).norm() / b.double().norm())  # noqa: E731
    assert rel(torch.stack(got), torch.stack(want)) < limit
    # the recurrent layer's tokens are those of one scan over prompt and tokens
    full, _ = scan.scan_fwd(torch.cat([x[:, :, :B * L].view(B, 1, L, D), rows(x).permute(1, 2, 0, 3)], 2).contiguous(),
                            torch.cat([z[:, :, :B * L].view(B, 1, L, D), rows(z).permute(1, 2, 0, 3)], 2).contiguous(),
                            write="leak", gate="preact", tau=TAU)
    assert rel(torch.stack(vs, 2).reshape(B, H, T, V), full[:, :, L:].view(B, T, H, V).transpose(1, 2)) < 2.0 ** -8
    # resume: the cached state (and window) as the h0 of a prefill
    back = gc.cache_load(c, slots, lengths)
    assert rel(back, S) < limit
    o1, _ = gla.gla_fwd(part(q, 0, L), part(k, 0, L), v, part(la, 0, L), back)
    o2, _ = gla.gla_fwd(part(q, 0, L), part(k, 0, L), v, part(la, 0, L), S)
    assert rel(o1, o2) < limit


@pytest.mark.gpu
def test_cache_checks(lib):
    c, S, g = fill_pool(3, 1, 32, 64, 4, "int8", torch.float32)
    slots, lengths = pool_case(c, [2, 0], [0, 1])
    t = {n: x.cuda() for n, x in token(c, 2, g).items()}
    gc.cache_store(c, S[:2].cuda(), slots, checks=True)
    gc.cache_step(c, t["q"], t["k"], t["v"], t["log_a"], slots, lengths, checks=True)
    gc.cache_load(c, slots, lengths, checks=True)
    t["log_a"][1, 0, 3] = 0.25
    with pytest.raises(gla.GlaError):
        gc.cache_step(c, t["q"], t["k"], t["v"], t["log_a"], slots, lengths, checks=True)


# ---------------------------------------------------------------- refusals (no GPU needed)


def _desc(**kw):
    d = dict(B=2, H=1, L=1, Dk=64, Dv=64, dtype=0, chunk=0, subchunk=0, state_mode=0, impl=0, flags=0, gate=0,
             gate_tau=0.0)
    d.update(kw)
    return _lib.GlaDesc(**d)


def _pool(**kw):
    d = dict(codes=16, scale=16, k=16, v=16, log_a=16, slots=4, window=16, format=0)
    d.update(kw)
    return _lib.GlaCache(**d)


def _all(lib, d, c):
    d, c = ctypes.byref(d), ctypes.byref(c)
    return (lib.gla_cache_store(d, c, 16, 16, None), lib.gla_cache_load(d, c, 16, 16, 16, None),
            lib.gla_cache_step(d, c, 16, 16, 16, 16, 16, 16, 16, None))


@pytest.mark.parametrize("bad,want", [(dict(B=0), 1), (dict(H=0), 1), (dict(Dk=0), 1), (dict(Dv=-3), 1), (dict(dtype=2), 1),
                                      (dict(flags=1), 1), (dict(gate=7), 1), (dict(gate=3), 1), (dict(chunk=64), 2),
                                      (dict(impl=2), 2), (dict(Dk=4096), 2), (dict(B=1 << 30), 2)])
def test_cache_bad_descriptor(lib, bad, want):
    assert _all(lib, _desc(**bad), _pool()) == (want,) * 3


@pytest.mark.parametrize("bad", [dict(slots=0), dict(slots=1 << 32), dict(window=0), dict(window=65), dict(format=2),
                                 dict(codes=None), dict(codes=24), dict(scale=None)])
def test_cache_bad_pool(lib, bad):
    assert _all(lib, _desc(), _pool(**bad)) == (1,) * 3


def test_cache_bad_pointers(lib):
    d = ctypes.byref(_desc())
    for n in ("k", "v", "log_a"):
        for p in (None, 20):
            c = ctypes.byref(_pool(**{n: p}))
            assert lib.gla_cache_load(d, c, 16, 16, 16, None) == 1
            assert lib.gla_cache_step(d, c, 16, 16, 16, 16, 16, 16, 16, None) == 1
    c = ctypes.byref(_pool())
    assert lib.gla_cache_store(None, c, 16, 16, None) == 1 and lib.gla_cache_store(d, None, 16, 16, None) == 1
    for p in (None, 18):
        assert lib.gla_cache_store(d, c, 16, p, None) == 1
        assert lib.gla_cache_load(d, c, p, 16, 16, None) == 1
        assert lib.gla_cache_step(d, c, 16, 16, 16, 16, 16, p, 16, None) == 1
    for i in list(range(4)) + [6]:
        a = [16] * 7
        a[i] = 8
        assert lib.gla_cache_step(d, c, *a, None) == 1, i
    assert lib.gla_cache_store(d, c, 8, 16, None) == 1
    assert lib.gla_cache_load(d, c, 16, 16, None, None) == 1


def test_cache_binding_refuses(lib):
    mk = lambda **kw: gc.StateCache.empty(4, 1, 8, 16, device="cpu", **kw)  # noqa: E731
    c = mk(window=2)
    s = torch.zeros(2, dtype=torch.int32)
    q, v, la = torch.zeros(2, 1, 8, dtype=torch.bfloat16), torch.zeros(2, 1, 16, dtype=torch.bfloat16), torch.zeros(2, 1, 8)
    with pytest.raises(ValueError):
        mk(format="int4")
    with pytest.raises(TypeError):
        mk(dtype=torch.float16)
    with pytest.raises(TypeError):
        gc.StateCache(c.codes.float(), c.scale, c.k, c.v, c.log_a)
    with pytest.raises(ValueError):
        gc.StateCache(c.codes, c.scale[..., :0], c.k, c.v, c.log_a)
    with pytest.raises(ValueError):
        gc.StateCache(c.codes.transpose(2, 3), c.scale, c.k, c.v, c.log_a)
    with pytest.raises(TypeError):
        gc.cache_store(c.codes, torch.zeros(2, 1, 8, 16), s)
    with pytest.raises(ValueError):
        gc.cache_store(c, torch.zeros(3, 1, 8, 16), s)
    with pytest.raises(TypeError):
        gc.cache_store(c, torch.zeros(2, 1, 8, 16), s.long())
    with pytest.raises(ValueError):
        gc.cache_load(c, s, s[:1])
    with pytest.raises(TypeError):
        gc.cache_step(c, q.float(), q, v, la, s, s)
    with pytest.raises(ValueError):
        gc.cache_step(c, q, q, v[..., :8], la, s, s)
    with pytest.raises(ValueError):
        gc.cache_step(c, q, q, v, la[..., 0], s, s)
    with pytest.raises(TypeError):
        gc.cache_step(c, q, q, v, la, s, None)
