"""Workloads of the gated linear recurrence (scan) and of the recurrent-state cache.

Each case names one pass through an operator. `run` computes it in plain torch operations (fp32), or, with
`own` set, through the package's entry points; `exact` computes the same outputs in fp64 from the definition,
token by token. Shapes come from the package's named layers (340M layer: B=8, H=4, L=2048, 128 x 256, width
1024; 1.3B layer: B=4, H=4, L=2048, 256 x 512, width 2048; long sequence: L=16384; decode: B=64) and from
ragged and odd sizes around them.
"""
import math

import torch

own = False

GROUP = 128  # state columns that share one scale


def listed():
    return [
        # --- scan forward: the smallest named workload, where the launch counts
        dict(name="scan_fwd_short", op="fwd", B=1, H=1, L=256, D=64, dtype="f32", gate="channel", write="input",
             packed=False, z_mean=0.0),
        # prefill of the 340M layer's width, eight sequences
        dict(name="scan_fwd_340m", op="fwd", B=8, H=1, L=2048, D=1024, dtype="bf16", gate="channel", write="leak",
             packed=False, z_mean=0.0),
        # ragged prefill: 23 prompts packed into one row axis with padding rows behind them, odd width
        dict(name="scan_fwd_packed", op="fwd", B=23, H=1, L=9973, D=777, dtype="bf16", gate="preact", write="leak",
             packed=True, z_mean=2.0),
        # --- scan training step (forward and backward): a small odd packed batch in fp32
        dict(name="scan_train_packed", op="train", B=5, H=2, L=1111, D=129, dtype="f32", gate="channel", write="input",
             packed=True, z_mean=0.0),
        # the 1.3B layer's width, gate given by its pre-activation
        dict(name="scan_train_1p3b", op="train", B=4, H=1, L=2048, D=2048, dtype="bf16", gate="preact", write="leak",
             packed=False, z_mean=0.0),
        # one long sequence with slow decay: little parallelism outside the time axis
        dict(name="scan_train_long", op="train", B=1, H=4, L=16384, D=256, dtype="bf16", gate="channel", write="input",
             packed=False, z_mean=2.0),
        # --- one token: a single stream, and a serving batch drawn from a pool of slots
        dict(name="scan_step_1", op="step", B=1, H=1, P=8, D=1024, dtype="bf16", gate="channel", write="input",
             z_mean=0.0),
        dict(name="scan_step_256", op="step", B=256, H=1, P=320, D=2048, dtype="bf16", gate="preact", write="leak",
             z_mean=2.0),
        # --- state cache: prompts' final states written into their slots
        dict(name="cache_store_64", op="store", B=64, H=4, P=96, K=128, V=256, W=16, fmt="e4m3", dtype="bf16"),
        # suspended sequences read back in the middle of their windows
        dict(name="cache_load_32", op="load", B=32, H=4, P=48, K=256, V=512, W=16, fmt="int8", dtype="bf16"),
        # decode of the named batch, one sixteenth of the rows folding their window
        dict(name="cache_step_64", op="cstep", B=64, H=4, P=96, K=128, V=256, W=16, fmt="e4m3", dtype="bf16",
             gate="channel", fold=True),
        # a large serving batch at the 1.3B layer's state size, none of the rows at its window's end
        dict(name="cache_step_256", op="cstep", B=256, H=4, P=288, K=256, V=512, W=16, fmt="int8", dtype="bf16",
             gate="preact", fold=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "train", "train", "step", "store", "load", "cstep", "cstep"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("fwd", "train"):
        packed = rng.random() < 0.4
        H = rng.choice([1, 1, 2, 4])
        D = _log_int(rng, 16, 4096 // H)
        B = _log_int(rng, 1, 16)
        L = _log_int(rng, 1, 16384)
        cost = H * L * D * (1 if packed else B) * (1 if dtype == "bf16" else 2)
        if cost > 16_000_000:
            L = max(1, L * 16_000_000 // cost)
        return dict(op=op, B=B, H=H, L=L, D=D, dtype=dtype, gate=rng.choice(["channel", "preact"]),
                    write=rng.choice(["input", "leak"]), packed=packed, z_mean=rng.choice([0.0, 2.0]))
    if op == "step":
        B = _log_int(rng, 1, 256)
        return dict(op=op, B=B, H=rng.choice([1, 4]), P=B + rng.randint(0, 64), D=_log_int(rng, 16, 1024), dtype=dtype,
                    gate=rng.choice(["channel", "preact"]), write=rng.choice(["input", "leak"]),
                    z_mean=rng.choice([0.0, 2.0]))
    B = _log_int(rng, 1, 64)
    K = rng.choice([16, 64, 96, 128, 256, rng.randint(8, 256)])
    V = rng.choice([64, 128, 256, 512, 16 * rng.randint(1, 32), rng.randint(8, 512)])
    H = rng.choice([1, 2, 4, 8])
    B = max(1, min(B, (1 << 24) // (H * K * V)))
    fmt = rng.choice(["int8", "e4m3"])
    c = dict(op=op, B=B, H=H, P=B + rng.randint(0, 16), K=K, V=V,
             W=rng.choice([4, 8, 16, 16, 32]), fmt=fmt, dtype=dtype)
    if op == "cstep":
        c.update(gate=rng.choice(["channel", "preact"]), fold=fmt == "e4m3")
    return c


TAU = 16.0
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _gen(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 17)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _slots(g, B, P):
    return torch.randperm(P, generator=g, device="cuda")[:B].to(torch.int32)


def _gates(case, g, *shape):
    z = _randn(g, *shape) + case.get("z_mean", 0.0)
    return z if case["gate"] == "preact" else torch.nn.functional.logsigmoid(z) / TAU


def _kinds(case):
    """The gate and write options as the calls take them."""
    return dict(write=case["write"], gate=case["gate"], tau=TAU if case["gate"] == "preact" else 0.0)


def prepare(case, seed):
    g, dt, op = _gen(case, seed), DT[case["dtype"]], case["op"]
    s = {"case": case}
    if op in ("fwd", "train"):
        B, H, L, D = case["B"], case["H"], case["L"], case["D"]
        lead = (1, H, L) if case["packed"] else (B, H, L)
        s["x"] = _randn(g, *lead, D).to(dt)
        s["log_a"] = _gates(case, g, *lead, D)
        s["h0"] = _randn(g, B, H, D)
        s["h"] = torch.zeros(*lead, D, dtype=dt, device="cuda")
        s["cu"] = None
        if case["packed"]:  # B prompts of random lengths, empty ones among them, and padding rows behind the last
            used = L - min(L - 1, L // 50)
            cuts = torch.sort(torch.randint(0, used + 1, (B - 1,), generator=g, device="cuda")).values
            ends = torch.tensor([0, used], device="cuda")
            s["cu"] = torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)
        if op == "train":
            s["dh"] = _randn(g, *lead, D).to(dt)
            s["dhT"] = _randn(g, B, H, D)
            s["out"] = {"dx": torch.zeros_like(s["x"]), "dlog_a": torch.zeros_like(s["log_a"])}
    elif op == "step":
        B, H, P, D = case["B"], case["H"], case["P"], case["D"]
        s["x"] = _randn(g, B, H, D).to(dt)
        s["log_a"] = _gates(case, g, B, H, D)
        s["state"] = _randn(g, P, H, D)
        s["slots"] = _slots(g, B, P)
    else:
        B, H, P, K, V, W = (case[n] for n in ("B", "H", "P", "K", "V", "W"))
        s["slots"] = _slots(g, B, P)
        rows = torch.rand(P, H, K, 1, generator=g, device="cuda") * 0.9 + 0.1  # rows of slow and of fast channels
        if op == "store":
            s["S"] = _randn(g, B, H, K, V) * rows[:B]
            codes, scale = _quantise(_randn(g, 1, 1, K, V).expand(P, H, K, V), case["fmt"])
        else:
            codes, scale = _quantise(_randn(g, P, H, K, V) * rows, case["fmt"])
        s["codes"], s["scale"] = codes, scale
        s["kw"] = (_randn(g, P, H, W, K) / K**0.5).to(dt)
        s["vw"] = (_randn(g, P, H, W, V) / K**0.5).to(dt)
        s["gw"] = torch.nn.functional.logsigmoid(_randn(g, P, H, W, K)) / TAU
        if op != "store":
            # tokens since the state was written; every fill of the window alike, without the last one where no
            # row folds
            n = torch.arange(B, device="cuda") % (W if op == "load" or case["fold"] else max(1, W - 1))
            s["lengths"] = (n + W * (torch.arange(B, device="cuda") % 3))[
                torch.randperm(B, generator=g, device="cuda")].to(torch.int32)
        if op == "cstep":
            s["q"] = (_randn(g, B, H, K) / K**0.5).to(dt)
            s["k"] = (_randn(g, B, H, K) / K**0.5).to(dt)
            s["v"] = (_randn(g, B, H, V) / K**0.5).to(dt)
            s["log_a"] = _gates(case, g, B, H, K)
    return s


# ---------------------------------------------------------------- plain forms


def _alpha(case, g):
    """(log a, a, w) of the gate argument."""
    la = torch.nn.functional.logsigmoid(g) / TAU if case["gate"] == "preact" else g
    return la, torch.exp(la), (-torch.expm1(la) if case["write"] == "leak" else torch.ones_like(la))


def _doubling(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 2 from zero: log2(L) passes that join spans of 1, 2, 4, ... steps."""
    d, L = 1, b.shape[2]
    while d < L:
        b = torch.cat([b[:, :, :d], torch.addcmul(b[:, :, d:], a[:, :, d:], b[:, :, :-d])], 2)
        a = torch.cat([a[:, :, :d], a[:, :, d:] * a[:, :, :-d]], 2)
        d *= 2
    return b


def _rows(s):
    """Per row: its sequence, whether it starts or ends it, and whether it belongs to one; dense rows as [1,1,L]."""
    x, cu = s["x"], s["cu"]
    t = torch.arange(x.shape[2], device=x.device)
    if cu is None:
        return None, (t == 0), (t == x.shape[2] - 1), torch.ones_like(t, dtype=torch.bool)
    n = torch.searchsorted(cu[1:], t, right=True, out_int32=False)
    ok = (n < cu.numel() - 1) & (t >= cu[0])
    n = n.clamp(max=cu.numel() - 2)
    return n, ok & (t == cu[n]), ok & (t == cu[n + 1] - 1), ok


def _plain_scan(s, train):
    case, x, cu = s["case"], s["x"].float(), s["cu"]
    la, a, w = _alpha(case, s["log_a"])
    n, start, end, ok = _rows(s)
    at = lambda h: h[:, :, None] if n is None else h[n].transpose(0, 1)[None]  # noqa: E731  [.,H,L|1,D]
    col = lambda m: m[None, None, :, None]  # noqa: E731
    h0 = at(s["h0"])
    a0 = torch.where(col(start) | ~col(ok), 0.0, a)
    b = torch.where(col(ok), w * x + torch.where(col(start), a * h0, 0.0), 0.0)
    h = _doubling(a0, b)
    s["h"].copy_(torch.where(col(ok), h, s["h"].float()))

    def last(z, empty):  # the value at each sequence's last row; empty sequences keep `empty`
        if n is None:
            return z[:, :, -1]
        e = (cu[1:] - 1).clamp(min=0).long()
        return torch.where((cu[1:] > cu[:-1])[:, None, None], z[0, :, e].transpose(0, 1), empty)

    out = [s["h"], last(h, s["h0"])]
    if train:
        r = s["dh"].float() + torch.where(col(end), at(s["dhT"]), 0.0)
        r = torch.where(col(ok), r, 0.0)
        # g_t = r_t + a_{t+1} g_{t+1}: the same passes over the reversed rows
        nxt = torch.cat([a[:, :, 1:], torch.zeros_like(a[:, :, :1])], 2)
        nxt = torch.where(col(end) | ~col(ok), 0.0, nxt)
        g = _doubling(nxt.flip(2), r.flip(2)).flip(2)
        hp = torch.where(col(start), h0, torch.cat([torch.zeros_like(h[:, :, :1]), h[:, :, :-1]], 2))
        dla = a * (hp - x if case["write"] == "leak" else hp) * g
        if case["gate"] == "preact":
            dla = dla * torch.sigmoid(-s["log_a"]) / TAU
        o = s["out"]
        o["dx"].copy_(torch.where(col(ok), w * g, o["dx"].float()))
        o["dlog_a"].copy_(torch.where(col(ok), dla, o["dlog_a"]))
        ag = a * g
        if n is None:
            dh0 = ag[:, :, 0]
        else:
            b0 = cu[:-1].clamp(max=x.shape[2] - 1).long()
            dh0 = torch.where((cu[1:] > cu[:-1])[:, None, None], ag[0, :, b0].transpose(0, 1), s["dhT"])
        out += [o["dx"], o["dlog_a"], dh0]
    return out


def _plain_step(s):
    _, a, w = _alpha(s["case"], s["log_a"])
    at = s["slots"].long()
    h = a * s["state"][at] + w * s["x"].float()
    s["state"].index_copy_(0, at, h)
    return [h.to(s["x"].dtype), s["state"]]


def _quantise(S, fmt):
    """8-bit codes and the scales of each row's groups of columns."""
    V = S.shape[-1]
    G = -(-V // GROUP)
    pad = torch.nn.functional.pad(S, (0, G * GROUP - V)).unflatten(-1, (G, GROUP))
    scale = pad.abs().amax(-1) * (1 / 127 if fmt == "int8" else 1 / 448)
    y = (pad * scale.reciprocal()[..., None]).flatten(-2)[..., :V]
    return (torch.round(y).clamp(-127, 127).to(torch.int8) if fmt == "int8" else y.to(torch.float8_e4m3fn)), scale


def _dequantise(codes, scale):
    return codes.float() * scale.repeat_interleave(GROUP, -1)[..., : codes.shape[-1]]


def _put(pool, at, rows):
    if pool.element_size() == 1:
        pool, rows = pool.view(torch.uint8), rows.contiguous().view(torch.uint8)
    pool.index_copy_(0, at, rows)


def _take(pool, at):
    return pool.view(torch.uint8)[at].view(pool.dtype) if pool.element_size() == 1 else pool[at]


def _windowed(s, at, kw, vw, gw, used):
    """State of each row: the cached state and its first `used` window tokens, later ones decayed less."""
    live = torch.arange(kw.shape[2], device=kw.device)[None, :] < used[:, None]
    gw = torch.where(live[:, None, :, None], gw, 0.0)
    later = torch.nn.functional.pad(gw[:, :, 1:], (0, 0, 0, 1)).flip(2).cumsum(2).flip(2)
    kt = torch.where(live[:, None, :, None], kw.float() * torch.exp(later), 0.0)
    S = _dequantise(_take(s["codes"], at), s["scale"][at]) * torch.exp(gw.sum(2))[..., None]
    return S + kt.transpose(2, 3) @ torch.where(live[:, None, :, None], vw.float(), 0.0)


def _plain_cache(s):
    case, at = s["case"], s["slots"].long()
    W = case["W"]
    if case["op"] == "store":
        codes, scale = _quantise(s["S"], case["fmt"])
        _put(s["codes"], at, codes)
        _put(s["scale"], at, scale)
        return [s["codes"], s["scale"]]
    n = s["lengths"].long() % W
    if case["op"] == "load":
        return [_windowed(s, at, s["kw"][at], s["vw"][at], s["gw"][at], n)]
    la = torch.nn.functional.logsigmoid(s["log_a"]) / TAU if case["gate"] == "preact" else s["log_a"]
    s["kw"][at, :, n] = s["k"]
    s["vw"][at, :, n] = s["v"]
    s["gw"][at, :, n] = la
    S = _windowed(s, at, s["kw"][at], s["vw"][at], s["gw"][at], n + 1)
    o = (s["q"].float()[:, :, None, :] @ S)[:, :, 0].to(s["q"].dtype)
    full = (n + 1 == W)[:, None, None, None]
    codes, scale = _quantise(S, case["fmt"])
    old = _take(s["codes"], at)
    _put(s["codes"], at, torch.where(full, codes.view(torch.uint8), old.view(torch.uint8)).view(codes.dtype))
    _put(s["scale"], at, torch.where(full, scale, s["scale"][at]))
    return [o, s["codes"], s["scale"], s["kw"], s["vw"], s["gw"]]


# ---------------------------------------------------------------- the package's calls

_own = {}


def _mods():
    if not _own:
        from chunkwise_linear_rnn_gla_b200 import cache, scan

        _own.update(cache=cache, scan=scan)
    return _own["scan"], _own["cache"]


def _own_run(s):
    scan, cache = _mods()
    case = s["case"]
    op = case["op"]
    if op == "fwd":
        h, hT = scan.scan_fwd(s["x"], s["log_a"], s["h0"], cu_seqlens=s["cu"], h=s["h"], **_kinds(case))
        return [h, hT]
    if op == "train":
        if "ws" not in s:
            s["ws"] = scan.scan_workspace(s["x"], s["cu"])
        h, hT = scan.scan_fwd(s["x"], s["log_a"], s["h0"], cu_seqlens=s["cu"], h=s["h"], workspace=s["ws"],
                              **_kinds(case))
        d = scan.scan_bwd(s["x"], s["log_a"], s["dh"], s["h0"], s["dhT"], cu_seqlens=s["cu"], workspace=s["ws"],
                          ws_from_fwd=True, out=s["out"], **_kinds(case))
        return [h, hT, d["dx"], d["dlog_a"], d["dh0"]]
    if op == "step":
        h = scan.scan_step(s["x"], s["log_a"], s["state"], s["slots"], **_kinds(case))
        return [h, s["state"]]
    if "cache" not in s:
        s["cache"] = cache.StateCache(s["codes"], s["scale"], s["kw"], s["vw"], s["gw"])
    c = s["cache"]
    if op == "store":
        cache.cache_store(c, s["S"], s["slots"])
        return [s["codes"], s["scale"]]
    if op == "load":
        return [cache.cache_load(c, s["slots"], s["lengths"])]
    o = cache.cache_step(c, s["q"], s["k"], s["v"], s["log_a"], s["slots"], s["lengths"], gate=case["gate"],
                         tau=TAU if case["gate"] == "preact" else 0.0)
    return [o, s["codes"], s["scale"], s["kw"], s["vw"], s["gw"]]


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    if op in ("fwd", "train"):
        return _plain_scan(state, op == "train")
    return _plain_step(state) if op == "step" else _plain_cache(state)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op in ("fwd", "train"):
        B, H, L, D = case["B"], case["H"], case["L"], case["D"]
        rows = H * ((L - min(L - 1, L // 50)) if case["packed"] else B * L)
        b = rows * D * (2 * e + 4) + 8 * B * H * D  # x, log_a, h; h0, hT
        f = rows * D * 4
        if op == "train":
            b += rows * D * (2 * e + 4) + 8 * B * H * D  # dh, dx, dlog_a; dhT, dh0
            f += rows * D * 8
        return {"bytes": b, "flops": f}
    B, H = case["B"], case["H"]
    if op == "step":
        return {"bytes": B * H * case["D"] * (2 * e + 12) + 4 * B, "flops": B * H * case["D"] * 4}
    K, V, W = case["K"], case["V"], case["W"]
    groups = -(-V // GROUP)
    entry = K * V + 4 * K * groups  # codes and scales of one head's state
    token = K * (e + 4) + V * e  # k, log a and v of one token
    if op == "store":
        return {"bytes": B * H * (4 * K * V + entry) + 4 * B, "flops": B * H * K * V * 3}
    if op == "load":
        fill = sum(i % W for i in range(B)) / B
        return {"bytes": B * H * (4 * K * V + entry + fill * token) + 8 * B, "flops": B * H * K * V * (2 + 2 * fill)}
    span = W if case["fold"] else max(1, W - 1)
    fill = sum(i % span for i in range(B)) / B
    folds = sum(i % span == W - 1 for i in range(B)) / B
    b = (1 + folds) * entry + fill * token + 2 * token + (K + V) * e  # the token is read and put into the window
    return {"bytes": B * H * b + 8 * B, "flops": B * H * (2 * K * V + (fill + 1) * (3 * K + 2 * V) + folds * 2 * W * K * V)}


# ---------------------------------------------------------------- fp64, from the definition, token by token


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    la = None
    if "log_a" in s:
        la = s["log_a"].double()
        if case["gate"] == "preact":
            la = -torch.log1p(torch.exp(-la)) / TAU
    if op in ("fwd", "train"):
        return _exact_scan(case, s, la)
    if op == "step":
        a = torch.exp(la)
        w = -torch.expm1(la) if case["write"] == "leak" else torch.ones_like(la)
        state = s["state"].double()
        h = a * state[s["slots"].long()] + w * s["x"].double()
        state[s["slots"].long()] = h
        return [h, state]
    fmt, V = case["fmt"], case["V"]
    of_col = torch.arange(V, device="cuda") // GROUP

    def quantise64(S):
        scale = torch.stack([S[..., of_col == i].abs().amax(-1) for i in range(int(of_col[-1]) + 1)], -1)
        scale = scale / (127 if fmt == "int8" else 448)
        y = S / scale[..., of_col]
        return (torch.round(y) if fmt == "int8" else y.float().to(torch.float8_e4m3fn)).double(), scale

    at = s["slots"].long()
    codes, scale = s["codes"].to(torch.float32).double() if op != "load" else None, s["scale"].double()
    if op == "store":
        codes[at], scale[at] = quantise64(s["S"].double())
        return [codes if fmt == "e4m3" else None, scale]
    S = _take(s["codes"], at).to(torch.float32).double() * scale[at][..., of_col]
    n = (s["lengths"].long() % case["W"]).tolist()
    kw, vw, gw = s["kw"].double(), s["vw"].double(), s["gw"].double()
    for i, b in enumerate(at.tolist()):
        for j in range(n[i]):
            S[i] = torch.exp(gw[b, :, j])[..., None] * S[i] + kw[b, :, j, :, None] * vw[b, :, j, None, :]
    if op == "load":
        return [S]
    k, v = s["k"].double(), s["v"].double()
    S = torch.exp(la)[..., None] * S + k[..., None] * v[:, :, None, :]
    o = (s["q"].double()[..., None] * S).sum(2)
    for i, b in enumerate(at.tolist()):
        kw[b, :, n[i]], vw[b, :, n[i]], gw[b, :, n[i]] = k[i], v[i], la[i]
        if n[i] + 1 == case["W"]:
            codes[b], scale[b] = quantise64(S[i])
    return [o, codes if fmt == "e4m3" else None, scale, kw, vw, gw]


def _exact_scan(case, s, la):
    x, a = s["x"].double(), torch.exp(la)
    w = -torch.expm1(la) if case["write"] == "leak" else torch.ones_like(la)
    T = x.shape[2]
    spans = [(0, T)] if s["cu"] is None else list(zip(s["cu"].tolist()[:-1], s["cu"].tolist()[1:]))
    pick = (lambda i: slice(None)) if s["cu"] is None else (lambda i: slice(i, i + 1))
    h, hT, before = torch.zeros_like(x), torch.zeros_like(s["h0"], dtype=torch.float64), torch.zeros_like(x)
    for i, (lo, hi) in enumerate(spans):
        y = s["h0"][pick(i)].double()
        for t in range(lo, hi):
            before[:, :, t] = y
            y = a[:, :, t] * y + w[:, :, t] * x[:, :, t]
            h[:, :, t] = y
        hT[pick(i)] = y
    if case["op"] == "fwd":
        return [h, hT]
    g, dh0, dh = torch.zeros_like(x), torch.zeros_like(hT), s["dh"].double()
    for i, (lo, hi) in enumerate(spans):
        y = s["dhT"][pick(i)].double()
        for t in range(hi - 1, lo - 1, -1):
            g[:, :, t] = dh[:, :, t] + y
            y = a[:, :, t] * g[:, :, t]
        dh0[pick(i)] = y
    dla = a * before * g - (a * x * g if case["write"] == "leak" else 0.0)
    if case["gate"] == "preact":
        dla = dla / (1 + torch.exp(s["log_a"].double())) / TAU
    return [h, hT, w * g, dla, dh0]
