"""The gated linear recurrence and the q/k norms with rotary positions: cases, inputs, plain forms.

`own` chooses what `run` computes with: this file's plain torch operations (False) or the library's kernels (True).

Gated linear recurrence ("lru"), per sequence and channel, on packed rows [T, D]:
    a_t = exp(g_t),  h_t = a_t h_{t-1} + b_t x_t,  o_t = h_t,
    b_t = 1 (gate "none"), 1 - a_t ("complement") or sqrt(1 - a_t^2) ("norm").
Its decode cache holds, per sequence and channel, the state S at the start of the current 32-token chunk and the
chunk's running composition (A, B), so that h = A S + B; a chunk that completes folds into S.

Norms of q and k with rotary positions ("qk"), per token and head, on x of d elements:
    z = x / sqrt(mean x^2 + eps) * (w_off + w)   (norm "rms"),  x / sqrt(sum x^2 + eps)  ("l2"),  x  ("none"),
    the first r elements of z turned in pairs by the angle pos * inv_freq_i, q times `scale`.
"""

import math

import torch

own = False

F32, BF16 = torch.float32, torch.bfloat16
DT = {"f32": F32, "bf16": BF16}
CHUNK = 32


def listed():
    lru = dict(D=4096, x="bf16", g="bf16", gate="norm", h0=True)
    qk = dict(Hq=16, Hk=16, d=128, r=128, inp="bf16", out="bf16", norm="l2", layout="half", fused=True, start=0)
    return [
        # one short prompt of a small model: the call's latency
        dict(lru, name="lru prefill 1x128", op="prefill", lens="128", D=2048, h0=False),
        # a rollout batch of equal prompts, decay kept in fp32
        dict(lru, name="lru prefill 4x2048", op="prefill", lens="2048x4", g="f32"),
        # a packed batch of very different prompts, with resets (g = -inf) between documents
        dict(lru, name="lru prefill 32 ragged", op="prefill", lens="128..8192x32", D=2048, gate="complement", reset=True),
        # token-by-token rollout, 64 sequences at mixed places of their chunks
        dict(lru, name="lru decode 64", op="decode", N=64),
        # a wide rollout batch, decay in fp32
        dict(lru, name="lru decode 1024", op="decode", N=1024, g="f32", gate="none"),
        # the trainer's step on a packed batch
        dict(lru, name="lru train 8x4096", op="train", lens="4096x8", g="f32"),
        # fp32 training of a few ragged sequences with an odd channel count
        dict(lru, name="lru train ragged f32", op="train", lens="1,777,2049,0,5003", D=1001, x="f32", g="f32", gate="none"),
        # one new token of 64 sequences, each at its own far position: weighted RMS norms, a quarter of the head turned
        dict(qk, name="qk decode 64", op="qk", T=64, Hq=32, Hk=8, d=256, r=64, norm="rms", start=200000, by_pos=True),
        # the rollout batch's q and k, slices of one projection, unit length and rotated
        dict(qk, name="qk prefill 4x2048", op="qk", lens="2048x4"),
        # a ragged batch continued at far positions: the rotation alone, neighbouring pairs
        dict(qk, name="qk rotate 32 ragged", op="qk", lens="128..8192x32", Hq=32, Hk=8, r=64, norm="none", layout="inter",
             start=100000, fused=False),
        # the trainer's gradient, with that of the norm's weights
        dict(qk, name="qk train 8x4096", op="qkgrad", lens="4096x8", norm="rms"),
        # fp32 gradients at an odd token count and a head size that is no power of two
        dict(qk, name="qk train odd f32", op="qkgrad", lens="1,333,0,1001", Hq=5, Hk=1, d=96, r=48, inp="f32", out="f32",
             norm="rms", layout="inter"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["prefill", "prefill", "decode", "train", "qk", "qk", "qkgrad"])
    if kind in ("prefill", "decode", "train"):
        c = dict(op=kind, D=_log(rng, 96, 5000), x=rng.choice(["bf16", "bf16", "f32"]), g=rng.choice(["bf16", "f32"]),
                 gate=rng.choice(["none", "complement", "norm"]), h0=rng.random() < 0.5)
        if kind == "decode":
            return dict(c, N=_log(rng, 1, 1024))
        n = _log(rng, 1, 32)
        most = min(16384, int((6e7 if kind == "train" else 1.5e8) / (n * c["D"])))
        lens = [_log(rng, 1, max(2, most)) for _ in range(n)]
        return dict(c, lens=",".join(map(str, lens)))
    d = rng.choice([16, 64, 80, 96, 128, 128, 192, 256])
    c = dict(op=kind, Hq=rng.choice([1, 3, 8, 16, 32]), Hk=rng.choice([1, 2, 8, 16]), d=d,
             r=rng.choice([d, d // 2, 16, 0]), inp=rng.choice(["bf16", "bf16", "f32"]), norm=rng.choice(["rms", "l2", "none"]),
             layout=rng.choice(["half", "inter"]), fused=rng.random() < 0.5, start=_log(rng, 1, 1000000))
    c["r"] -= c["r"] % 8
    c["out"] = rng.choice([c["inp"], "f32"])
    if kind == "qk" and rng.random() < 0.4:
        return dict(c, T=_log(rng, 1, 512), by_pos=True)
    n = _log(rng, 1, 24)
    most = max(2, int(1.2e8 / (n * (c["Hq"] + c["Hk"]) * d)))
    return dict(c, lens=",".join(str(_log(rng, 1, min(16384, most))) for _ in range(n)))


def _lens(case):
    """The sequence lengths: "7,0,9", "2048x4" (four of 2048) or "128..8192x32" (thirty-two, the same for every seed)."""
    s = case["lens"]
    if ".." in s:
        span, n = s.split("x")
        lo, hi = (int(v) for v in span.split(".."))
        gen = torch.Generator().manual_seed(4)
        return [int(v) for v in torch.randint(lo, hi + 1, (int(n),), generator=gen)]
    if "x" in s:
        length, n = s.split("x")
        return [int(length)] * int(n)
    return [int(v) for v in s.split(",")]


def _cu(lens):
    cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(lens, dtype=torch.int64), 0).to(torch.int32)
    return cu


def _log_decay(case, gen, shape):
    """g: a log decay per channel times a per-token gate for "norm" (decays of 0.9 .. 0.999 at an open gate), else -softplus."""
    z = torch.randn(shape, generator=gen, device="cuda")
    if case["gate"] == "norm":
        top = torch.log(torch.rand(shape[-1], generator=gen, device="cuda") * 0.099 + 0.9)
        g = top * torch.sigmoid(z)
    else:
        g = -torch.log1p(torch.exp(z))
    if case.get("reset"):
        g = torch.where(torch.rand(shape[0], 1, generator=gen, device="cuda") < 1e-3, float("-inf"), g)
    return g.to(DT[case["g"]])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    rn = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    s = {"case": case}
    if case["op"] == "decode":
        N, D = case["N"], case["D"]
        s["x"], s["g"] = rn(N, D).to(DT[case["x"]]), _log_decay(case, gen, (N, D))
        s["pos"] = torch.randint(0, CHUNK, (N, 1), generator=gen, device="cuda", dtype=torch.int32).repeat(1, -(-D // 256))
        s["S"], s["B"] = rn(N, D), rn(N, D)
        s["A"] = torch.rand(N, D, generator=gen, device="cuda")
        s["o"] = torch.empty_like(s["x"])
        if own:
            from linear_attention_rnn_gated_amd import binding as lib
            s["shape"] = lib.make_lru_shape(D, DT[case["x"]], DT[case["g"]], case["gate"])
            s["cache"] = lib.LruCache.of(s["S"], s["A"], s["B"], s["pos"])
        return s
    if case["op"] in ("prefill", "train"):
        lens, D = _lens(case), case["D"]
        s["lens"], s["cu_host"] = lens, _cu(lens)
        s["cu"] = s["cu_host"].cuda()
        T, N = sum(lens), len(lens)
        s["x"], s["g"] = rn(T, D).to(DT[case["x"]]), _log_decay(case, gen, (T, D))
        s["h0"] = 0.5 * rn(N, D) if case["h0"] else None
        if case["op"] == "train":
            s["do"], s["dhT"] = rn(T, D).to(DT[case["x"]]), rn(N, D)
        if own:
            from linear_attention_rnn_gated_amd import binding as lib
            s["shape"] = lib.make_lru_shape(D, DT[case["x"]], DT[case["g"]], case["gate"])
            if case["op"] == "train":
                s["ws"] = torch.empty(lib.lru_workspace_bytes(s["shape"], N, T), dtype=torch.uint8, device="cuda")
        return s
    Hq, Hk, d, r = case["Hq"], case["Hk"], case["d"], case["r"]
    if case.get("by_pos"):
        T = case["T"]
        s["pos"] = torch.randint(0, case["start"] + 1, (T,), generator=gen, device="cuda", dtype=torch.int32)
    else:
        lens = _lens(case)
        T, N = sum(lens), len(lens)
        s["lens"], s["cu"] = lens, _cu(lens).cuda()
        s["start"] = torch.randint(0, case["start"] + 1, (N,), generator=gen, device="cuda", dtype=torch.int32)
    dt, odt = DT[case["inp"]], DT[case["out"]]
    if case["fused"]:  # q and k are slices of one projection's rows, which hold v behind them
        row = rn(T, (Hq + 2 * Hk) * d).to(dt)
        s["q"], s["k"] = row[:, :Hq * d].unflatten(1, (Hq, d)), row[:, Hq * d:(Hq + Hk) * d].unflatten(1, (Hk, d))
    else:
        s["q"], s["k"] = rn(T, Hq, d).to(dt), rn(T, Hk, d).to(dt)
    if case["norm"] == "rms":
        s["w_q"], s["w_k"] = 0.1 * rn(d), 0.1 * rn(d)
    if case["op"] == "qkgrad":
        s["dq_out"], s["dk_out"] = rn(T, Hq, d).to(odt), rn(T, Hk, d).to(odt)
    # frequencies of a context stretched four times by linear scaling of the positions
    s["inv_freq"] = (10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / max(r, 1)) / 4).to(F32).cuda()
    s["scale"] = d ** -0.5
    if own:
        from linear_attention_rnn_gated_amd import binding as lib
        s["shape"] = lib.make_qk_shape(Hq, Hk, d, r, dt, out_dtype=odt, norm=case["norm"],
                                       layout="interleaved" if case["layout"] == "inter" else "half",
                                       eps=1e-6, scale=s["scale"], weight_offset=1.0)
        if case["op"] == "qkgrad":
            s["ws"] = torch.empty(lib.qk_workspace_bytes(s["shape"], T), dtype=torch.uint8, device="cuda")
    return s


# ---- the recurrence in plain operations -------------------------------------------------------------------------------


def _gated(case, x, g):
    """a = exp(g), the input's weight b, and b x, in fp32."""
    g = g.float()
    a = torch.exp(g)
    if case["gate"] == "none":
        b = torch.ones_like(a)
    elif case["gate"] == "complement":
        b = -torch.expm1(g)
    else:
        b = torch.sqrt(torch.clamp(-torch.expm1(2 * g), min=0))
    return a, b, b * x.float()


def _scan(a, u, longest):
    """h_t = a_t h_{t-1} + u_t down the rows, by doubling the span that each row's pair (a, u) covers."""
    span = 1
    while span < longest:
        u = torch.cat([u[:span], u[span:] + a[span:] * u[:-span]])
        a = torch.cat([a[:span], a[span:] * a[:-span]])
        span *= 2
    return u


def _ends(s):
    """First and last rows of the sequences that have any, and which those are."""
    cu = s["cu"].long()
    some = torch.nonzero(cu[1:] > cu[:-1]).flatten()
    return cu[:-1][some], cu[1:][some] - 1, some


def _h0(s):
    return s["h0"] if s["h0"] is not None else torch.zeros(len(s["lens"]), s["x"].shape[1], device="cuda")


def _plain_states(s):
    first, last, some = _ends(s)
    a, b, u = _gated(s["case"], s["x"], s["g"])
    h0 = _h0(s)
    u1, a1 = u.clone(), a.clone()
    u1[first] += a[first] * h0[some]
    a1[first] = 0
    h = _scan(a1, u1, max(s["lens"]))
    hT = h0.clone()
    hT[some] = h[last]
    return a, b, h, hT


def _plain_train(s):
    case, x = s["case"], s["x"].float()
    first, last, some = _ends(s)
    a, b, h, hT = _plain_states(s)
    up = s["do"].float().clone()
    up[last] += s["dhT"][some]
    nxt = torch.cat([a[1:], a[:1]])
    nxt[last] = 0
    d = _scan(nxt.flip(0), up.flip(0), max(s["lens"])).flip(0)
    prev = torch.cat([h[:1], h[:-1]])
    prev[first] = _h0(s)[some]
    dg = a * d * prev
    if case["gate"] == "complement":
        dg = dg - a * d * x
    elif case["gate"] == "norm":
        dg = dg - torch.where(b > 0, a * a / b, torch.zeros_like(b)) * d * x
    dh0 = s["dhT"].clone()
    dh0[some] = a[first] * d[first]
    return {"o": h.to(s["x"].dtype), "hT": hT, "dx": (b * d).to(s["x"].dtype), "dg": dg.to(s["g"].dtype), "dh0": dh0}


def _plain_decode(s):
    a, _, u = _gated(s["case"], s["x"], s["g"])
    A, B = a * s["A"], a * s["B"] + u
    h = A * s["S"] + B
    done = s["pos"][:, :1] == CHUNK - 1
    s["S"].copy_(torch.where(done, h, s["S"]))
    s["A"].copy_(torch.where(done, torch.ones_like(A), A))
    s["B"].copy_(torch.where(done, torch.zeros_like(B), B))
    s["pos"].copy_((s["pos"] + 1) % CHUNK)
    s["o"].copy_(h)


# ---- the norms and the rotation in plain operations -------------------------------------------------------------------


def _positions(s):
    if "pos" in s:
        return s["pos"].long()
    cu = s["cu"].long()
    n = torch.repeat_interleave(torch.arange(len(s["lens"]), device="cuda"), cu[1:] - cu[:-1])
    return torch.arange(int(s["q"].shape[0]), device="cuda") - cu[n] + s["start"].long()[n]


def _turn(s):
    angle = _positions(s).double()[:, None] * s["inv_freq"].double()
    return torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]


def _pairs(case, x):
    r = case["r"]
    if case["layout"] == "half":
        return x[..., :r // 2], x[..., r // 2:r], x[..., r:]
    return x[..., 0:r:2], x[..., 1:r:2], x[..., r:]


def _joined(case, lo, hi, rest):
    if case["layout"] == "half":
        return torch.cat([lo, hi, rest], -1)
    return torch.cat([torch.stack([lo, hi], -1).flatten(-2), rest], -1)


def _rotated(case, x, cos, sin):
    lo, hi, rest = _pairs(case, x)
    return _joined(case, lo * cos - hi * sin, hi * cos + lo * sin, rest)


def _inverse_norm(case, x):
    ss = (x * x).sum(-1, keepdim=True)
    return 1 / torch.sqrt((ss / case["d"] if case["norm"] == "rms" else ss) + 1e-6)


def _plain_qk(s, name, cos, sin):
    case, x = s["case"], s[name].float()
    if case["norm"] != "none":
        x = x * _inverse_norm(case, x)
    if case["norm"] == "rms":
        x = x * (1 + s["w_" + name])
    return (_rotated(case, x, cos, sin) * (s["scale"] if name == "q" else 1.0)).to(DT[case["out"]])


def _plain_qk_grad(s, name, cos, sin):
    case, x = s["case"], s[name].float()
    dz = _rotated(case, s["d%s_out" % name].float() * (s["scale"] if name == "q" else 1.0), cos, -sin)
    out = {}
    if case["norm"] != "none":
        inv = _inverse_norm(case, x)
        if case["norm"] == "rms":
            out["dw_" + name] = (dz * x * inv).sum((0, 1))
            dz = dz * (1 + s["w_" + name])
        n = case["d"] if case["norm"] == "rms" else 1
        dz = inv * (dz - x * (inv * inv / n * (dz * x).sum(-1, keepdim=True)))
    out["d" + name] = dz.to(x.dtype if case["inp"] == "f32" else BF16)
    return out


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        from linear_attention_rnn_gated_amd import binding as lib
        if op == "decode":
            lib.gdn_lru_decode_step(s["shape"], s["x"], s["g"], s["cache"], out=s["o"])
            return {"o": s["o"], "S": s["S"], "A": s["A"], "B": s["B"], "pos": s["pos"]}
        if op == "prefill":
            o, hT = lib.gdn_lru_prefill(s["shape"], s["x"], s["g"], s["cu"], h0=s["h0"], cu_seqlens_host=s["cu_host"])
            return {"o": o, "hT": hT}
        if op == "train":
            return lib.gdn_lru_fwd_bwd(s["shape"], s["x"], s["g"], s["cu"], s["do"], h0=s["h0"], dhT=s["dhT"], ws=s["ws"],
                                       cu_seqlens_host=s["cu_host"])
        at = {"pos": s["pos"]} if "pos" in s else {"cu_seqlens": s["cu"], "start": s["start"]}
        if op == "qk":
            qo, ko = lib.gdn_qk_rotary(s["shape"], s["q"], s["k"], s["inv_freq"], w_q=s.get("w_q"), w_k=s.get("w_k"), **at)
            return {"q": qo, "k": ko}
        return lib.gdn_qk_rotary_bwd(s["shape"], s["q"], s["k"], s["dq_out"], s["dk_out"], s["inv_freq"], w_q=s.get("w_q"),
                                     w_k=s.get("w_k"), ws=s["ws"], **at)
    if op == "decode":
        _plain_decode(s)
        return {"o": s["o"], "S": s["S"], "A": s["A"], "B": s["B"], "pos": s["pos"]}
    if op == "prefill":
        _, _, h, hT = _plain_states(s)
        return {"o": h.to(s["x"].dtype), "hT": hT}
    if op == "train":
        return _plain_train(s)
    cos, sin = _turn(s)
    if op == "qk":
        return {"q": _plain_qk(s, "q", cos, sin), "k": _plain_qk(s, "k", cos, sin)}
    return {**_plain_qk_grad(s, "q", cos, sin), **_plain_qk_grad(s, "k", cos, sin)}


def work(case):
    """Each input read once and each output written once; the operations of the formulas, an exp, a root or an angle as one."""
    size = {"f32": 4, "bf16": 2}
    if case["op"] == "decode":
        n = case["N"] * case["D"]
        # x, g and o, the state as one number per channel read and written
        return {"bytes": n * (2 * size[case["x"]] + size[case["g"]] + 8), "flops": n * 5}
    if case["op"] in ("prefill", "train"):
        lens = _lens(case)
        n, ends = sum(lens) * case["D"], len(lens) * case["D"] * 4
        if case["op"] == "prefill":
            return {"bytes": n * (2 * size[case["x"]] + size[case["g"]]) + ends * (2 if case["h0"] else 1), "flops": n * 5}
        return {"bytes": n * (4 * size[case["x"]] + 2 * size[case["g"]]) + ends * (4 if case["h0"] else 3), "flops": n * 12}
    T = case["T"] if case.get("by_pos") else sum(_lens(case))
    n = T * (case["Hq"] + case["Hk"]) * case["d"]
    if case["op"] == "qk":
        return {"bytes": n * (size[case["inp"]] + size[case["out"]]) + 4 * T, "flops": n * 8}
    return {"bytes": n * (2 * size[case["inp"]] + size[case["out"]]) + 4 * T, "flops": n * 14}


# ---- the definitions in 64 bits, token by token -----------------------------------------------------------------------


def _exact_lru(case, s):
    f = lambda t: None if t is None else t.double()  # noqa: E731
    T, D, N = s["x"].shape[0], case["D"], len(s["lens"])
    lens = torch.tensor(s["lens"])
    order = torch.argsort(lens, descending=True)  # at step t the sequences longer than t are the first ones
    length, first = lens[order].tolist(), s["cu"].long().cpu()[:-1][order].cuda()
    live = [sum(1 for v in length if v > t) for t in range(max(length))]
    order = order.cuda()

    def gate(t, n):
        g, x = f(s["g"][first[:n] + t]), f(s["x"][first[:n] + t])
        a = g.exp()
        b = {"none": lambda: torch.ones_like(a), "complement": lambda: -g.expm1(),
             "norm": lambda: (-(2 * g).expm1()).clamp(min=0).sqrt()}[case["gate"]]()
        return a, b, x

    state = f(s["h0"])[order].clone() if s["h0"] is not None else torch.zeros(N, D, dtype=torch.float64, device="cuda")
    begin = state.clone()
    h = torch.empty(T, D, dtype=torch.float64, device="cuda")
    for t, n in enumerate(live):
        a, b, x = gate(t, n)
        state[:n] = a * state[:n] + b * x
        h[first[:n] + t] = state[:n]
    out = {"o": h, "hT": torch.empty_like(state)}
    out["hT"][order] = state
    if case["op"] == "prefill":
        return out
    carry = f(s["dhT"])[order].clone()  # the gradient of the state behind step t
    dx, dg = torch.empty_like(h), torch.empty_like(h)
    for t in range(len(live) - 1, -1, -1):
        n = live[t]
        a, b, x = gate(t, n)
        before = h[first[:n] + t - 1] if t else begin[:n]
        dh = carry[:n] + f(s["do"][first[:n] + t])
        db = {"none": lambda: 0 * a, "complement": lambda: -a, "norm": lambda: torch.where(b > 0, -a * a / b, 0 * a)}[case["gate"]]()
        dx[first[:n] + t] = b * dh
        dg[first[:n] + t] = dh * (a * before + db * x)
        carry[:n] = a * dh
    out.update(dx=dx, dg=dg, dh0=torch.empty_like(carry))
    out["dh0"][order] = carry
    return out


def _exact_decode(case, s):
    g, x = s["g"].double(), s["x"].double()
    a = g.exp()
    b = {"none": 1.0, "complement": -g.expm1(), "norm": (-(2 * g).expm1()).clamp(min=0).sqrt()}[case["gate"]]
    S, A, B = s["S"].double().clone(), a * s["A"].double(), a * s["B"].double() + b * x
    h = A * S + B
    full = (s["pos"][:, 0] == CHUNK - 1).nonzero().flatten()
    S[full], A[full], B[full] = h[full], 1.0, 0.0
    return {"o": h, "S": S, "A": A, "B": B, "pos": (s["pos"] + 1) % CHUNK}


def _exact_qk(case, s):
    d, r = case["d"], case["r"]
    if "pos" in s:
        pos = s["pos"].double()
    else:
        pos = torch.cat([torch.arange(n, dtype=torch.float64, device="cuda") + float(p) for n, p in zip(s["lens"], s["start"].tolist())])
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"), pos[:, None] * s["inv_freq"].double()[None])[:, None]
    out = {}
    for name in ("q", "k"):
        x = s[name].double().detach().requires_grad_(case["op"] == "qkgrad")
        w = s["w_" + name].double().requires_grad_(case["op"] == "qkgrad") if case["norm"] == "rms" else None
        z = x
        if case["norm"] == "rms":
            z = x * ((x.square().mean(-1, keepdim=True) + 1e-6) ** -0.5) * (1.0 + w)
        elif case["norm"] == "l2":
            z = x * ((x.square().sum(-1, keepdim=True) + 1e-6) ** -0.5)
        if r:
            part = z[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2) if case["layout"] == "half" else z[..., :r].unflatten(-1, (r // 2, 2))
            part = torch.view_as_real(torch.view_as_complex(part.contiguous()) * turn)
            part = part.transpose(-1, -2).flatten(-2) if case["layout"] == "half" else part.flatten(-2)
            z = torch.cat([part, z[..., r:]], -1)
        y = z * s["scale"] if name == "q" else z
        if case["op"] == "qk":
            out[name] = y
            continue
        got = torch.autograd.grad(y, [x] if w is None else [x, w], s["d%s_out" % name].double())
        out["d" + name] = got[0]
        if w is not None:
            out["dw_" + name] = got[1]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "decode":
        return _exact_decode(case, s)
    return _exact_lru(case, s) if case["op"] in ("prefill", "train") else _exact_qk(case, s)
