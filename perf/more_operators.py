"""Causal attention, its gradient, the 8-bit key/value cache and attention over it: cases, inputs, plain forms.

`own` chooses what `run` computes with: this file's plain torch operations (False) or the library's kernels (True).

Attention ("attn", "train"), per query head h and the key/value head h / (Hq / Hkv), on packed rows [T, H, d]:
    s_ij = scale q_i . k_j  (j <= i),  p = softmax_j(s),  o_i = sum_j p_ij v_j,  lse_i = log sum_j exp(s_ij).

The cache ("write", "read", "decode"): keys and values in e4m3, in pages of P tokens [pages, Hkv, P, d]; every 32 tokens
of a head (k and v apart) share a scale, the least power of two s with max |x| / s <= 448.  Sequence n's token t is in
page block_table[n, t / P].  A block that gets more tokens keeps the larger scale; its older codes go over to it.
"""

import math

import torch

own = False

DEV = "cuda"
F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
DT = {"f32": F32, "bf16": BF16}
BLOCK = 32
LEAST = 2.0 ** -117


def listed():
    a = dict(Hq=32, Hkv=8, d=128, t="bf16")
    hybrid = dict(Hq=16, Hkv=2, d=256, t="bf16")
    return [
        # one short prompt: the call's latency
        dict(hybrid, name="attn prefill 1x128", op="attn", lens="128"),
        # a rollout batch of equal prompts
        dict(a, name="attn prefill 4x2048", op="attn", lens="2048x4"),
        # a packed batch of very different prompts; q, k and v are slices of one projection's rows
        dict(hybrid, name="attn prefill 32 ragged", op="attn", lens="128..8192x32", fused=True),
        # the trainer's step on a packed batch
        dict(a, name="attn train 8x4096", op="train", lens="4096x8"),
        # fp32 training of a few ragged sequences, one of them empty
        dict(name="attn train ragged f32", op="train", Hq=6, Hkv=2, d=64, t="f32", lens="1,777,2049,0,1003"),
        # one new token of 64 sequences, each somewhere in a block
        dict(a, name="kv write decode 64", op="write", new="1x64", old="1..4000x64", P=64),
        # the prompts of a ragged batch into fresh pages
        dict(a, name="kv write 32 ragged", op="write", new="128..8192x32", old="0x32", P=64),
        # cached prompts back in the type of the activations
        dict(hybrid, name="kv read 16 ragged", op="read", new="128..8192x16", old="0x16", P=128),
        # a token of each of a few sequences that have just begun
        dict(hybrid, name="attn decode 4 short", op="decode", new="1x4", old="1..100x4", P=64),
        # token-by-token rollout, 64 sequences of mixed lengths
        dict(a, name="attn decode 64", op="decode", new="1x64", old="128..8192x64", P=64),
        # one sequence with a long history
        dict(hybrid, name="attn decode 1 long", op="decode", new="1", old="131071", P=256),
        # the next parts of eight prompts whose beginnings are cached
        dict(a, name="attn continue 8", op="decode", new="64..500x8", old="500..8192x8", P=64, fused=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "train", "write", "read", "decode", "decode", "decode"])
    hkv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, Hq=hkv * rng.choice([1, 2, 3, 4, 8]), Hkv=hkv, d=rng.choice([64, 128, 128, 256]),
             t=rng.choice(["bf16", "bf16", "bf16", "f32"]))
    if op in ("attn", "train"):
        n = _log(rng, 1, 32)
        # pairs x heads x d within the listed cases'
        cost = {"attn": 8e11, "train": 2e11}[op] * (0.1 if c["t"] == "f32" else 1)
        most = min(16384, int(math.sqrt(cost / (n * c["Hq"] * c["d"]))))
        lens = [_log(rng, 1, max(2, most)) for _ in range(n)]
        return dict(c, lens=",".join(map(str, lens)), fused=rng.random() < 0.5)
    c.update(P=rng.choice([32, 64, 96, 256]), fused=rng.random() < 0.5)
    n = _log(rng, 1, 256)
    most = max(40, min(60000, int(3e8 / (n * hkv * c["d"]))))
    old = [_log(rng, 1, most) - 1 for _ in range(n)]
    if op == "decode" and rng.random() < 0.7:
        new = [1] * n
    else:
        cap = max(2, min(2000, int(3e7 / (n * c["Hq"] * c["d"])))) if op == "decode" else most
        new = [_log(rng, 1, cap) for _ in range(n)]
        if op == "decode":  # pairs of the padded plain form
            worst = max(2, int(2e9 / (n * c["Hq"] * max(new))))
            old = [min(v, worst) for v in old]
    return dict(c, new=",".join(map(str, new)), old=",".join(map(str, old)))


def _lens(s, salt=4):
    """Lengths: "7,0,9", "2048x4" (four of 2048) or "128..8192x32" (thirty-two, the same for every seed)."""
    if ".." in s:
        span, n = s.split("x")
        lo, hi = (int(v) for v in span.split(".."))
        gen = torch.Generator().manual_seed(salt)
        return [int(v) for v in torch.randint(lo, hi + 1, (int(n),), generator=gen)]
    if "x" in s:
        length, n = s.split("x")
        return [int(length)] * int(n)
    return [int(v) for v in s.split(",")]


def _cu(lens):
    cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(lens, dtype=torch.int64), 0).to(torch.int32)
    return cu


def _owner(lens):
    """For each packed row its sequence and its place there."""
    n = torch.tensor(lens, device=DEV)
    seq = torch.repeat_interleave(torch.arange(len(lens), device=DEV), n)
    first = torch.cumsum(n, 0) - n
    return seq, torch.arange(int(seq.numel()), device=DEV) - first[seq]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    rn = lambda *shape: torch.randn(*shape, generator=gen, device=DEV)  # noqa: E731
    Hq, Hkv, d, dt = case["Hq"], case["Hkv"], case["d"], DT[case["t"]]
    s = {"case": case, "scale": d ** -0.5}
    # keys and queries as per-head norms with weights leave them: a few channels larger than the rest
    w = 1 + 0.3 * rn(d)
    w[torch.randint(0, d, (3,), generator=gen, device=DEV)] *= 3

    def rows(T):
        q, k, v = rn(T, Hq, d), rn(T, Hkv, d) * w, rn(T, Hkv, d)
        if case.get("fused"):  # slices of one projection's rows
            row = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1)], 1).to(dt)
            return [x.unflatten(1, (-1, d)) for x in row.split([Hq * d, Hkv * d, Hkv * d], 1)]
        return [q.to(dt), k.to(dt), v.to(dt)]

    if case["op"] in ("attn", "train"):
        s["lens"] = _lens(case["lens"])
        s["cu"] = _cu(s["lens"]).to(DEV)
        T = sum(s["lens"])
        s["q"], s["k"], s["v"] = rows(T)
        if case["op"] == "train":
            s["do"] = rn(T, Hq, d).to(dt)
        if own:
            from linear_attention_rnn_gated_amd import binding as lib
            s["shape"] = lib.make_attn_shape(Hq, Hkv, d, dt, scale=s["scale"])
            if case["op"] == "train":
                s["ws"] = torch.empty(lib.attn_workspace_bytes(s["shape"], T, T), dtype=torch.uint8, device=DEV)
        return s

    P, old, new = case["P"], _lens(case["old"], 5), _lens(case["new"])
    whole = [a + b for a, b in zip(old, new)]
    n, T = len(new), sum(new)
    per = [-(-v // P) for v in whole]
    pages = sum(per) + 3
    # each sequence's pages lie anywhere in the pool; places of the table that hold no page are -1
    table = torch.full((n, max(per)), -1, dtype=torch.int32, device=DEV)
    own_page = torch.arange(max(per), device=DEV) < torch.tensor(per, device=DEV)[:, None]
    table[own_page] = torch.randperm(pages, generator=gen, device=DEV)[:sum(per)].to(torch.int32)
    s.update(old=old, new=new, whole=whole, table=table)
    # what the pool held before: any codes, NaN among them where they are not returned
    top = 127 if case["op"] == "write" else 128
    s["kc"], s["vc"] = (((torch.randint(0, top, (pages, Hkv, P, d), generator=gen, device=DEV, dtype=torch.uint8)
                          + 128 * torch.randint(0, 2, (pages, Hkv, P, d), generator=gen, device=DEV, dtype=torch.uint8)))
                        .view(E4M3) for _ in range(2))
    s["ks"], s["vs"] = (torch.full((pages, Hkv, P // BLOCK), 2.0 ** -8, device=DEV) for _ in range(2))
    held = old if case["op"] == "write" else whole
    if sum(held):
        hk, hv = (rn(sum(held), Hkv, d) * w).to(dt), rn(sum(held), Hkv, d).to(dt)
        _plain_write(s, hk, hv, held, [0] * n)
    s["cu"], s["start"] = _cu(new).to(DEV), torch.tensor(old, dtype=torch.int32, device=DEV)
    s["len"] = torch.tensor(whole, dtype=torch.int32, device=DEV)
    s["one"] = max(new) == min(new) == 1
    if case["op"] != "read":
        s["q"], s["k"], s["v"] = rows(T)
    if own:
        from linear_attention_rnn_gated_amd import binding as lib
        s["shape"] = lib.make_attn_shape(Hq, Hkv, d, dt, scale=s["scale"])
        s["cache"] = lib.KvCache.of(s["kc"], s["ks"], s["vc"], s["vs"])
        if case["op"] == "decode":
            s["ws"] = torch.empty(lib.attn_decode_workspace_bytes(s["shape"], n, T, max(whole)), dtype=torch.uint8,
                                  device=DEV)
    return s


# ---- attention in plain operations ------------------------------------------------------------------------------------


def _scores(s, q, k):
    """Scaled scores [Hkv, G, L, L] of one sequence, -inf above the diagonal."""
    L, Hkv, d = k.shape
    qg = q.float().unflatten(1, (Hkv, -1)).permute(1, 2, 0, 3).reshape(Hkv, -1, d)
    x = torch.matmul(qg, k.float().permute(1, 2, 0).contiguous()).view(Hkv, -1, L, L) * s["scale"]
    i = torch.arange(L, device=DEV)
    return qg, torch.where(i[None, :] <= i[:, None], x, float("-inf"))


def _softmax(x):
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(-1, keepdim=True)
    return e / z, (m + torch.log(z)).squeeze(-1)


def _rows(x, Hkv, L):
    """[Hkv, G L, d] as [L, Hq, d]."""
    return x.view(Hkv, -1, L, x.shape[-1]).permute(2, 0, 1, 3).flatten(1, 2)


def _plain_attn(s):
    q, dt, (T, Hkv, d) = s["q"], s["q"].dtype, s["k"].shape
    o = torch.empty(T, q.shape[1], d, dtype=dt, device=DEV)
    lse = torch.empty(T, q.shape[1], device=DEV)
    out = {"o": o, "lse": lse}
    if "do" in s:
        out.update(dq=torch.empty_like(o), dk=torch.empty(T, Hkv, d, dtype=dt, device=DEV),
                   dv=torch.empty(T, Hkv, d, dtype=dt, device=DEV))
    at = 0
    for L in s["lens"]:  # a sequence at a time: no pairs across sequences
        here = slice(at, at + L)
        at += L
        if L == 0:
            continue
        k, v = s["k"][here], s["v"][here].float().transpose(0, 1).contiguous()
        qg, x = _scores(s, q[here], k)
        p, z = _softmax(x)
        del x
        y = torch.matmul(p.view(Hkv, -1, L), v)
        o[here] = _rows(y, Hkv, L).to(dt)
        lse[here] = z.permute(2, 0, 1).flatten(1)
        if "do" in s:
            kk = k.float().transpose(0, 1).contiguous()
            do = s["do"][here].float().unflatten(1, (Hkv, -1)).permute(1, 2, 0, 3).reshape(Hkv, -1, d)
            p = p.view(Hkv, -1, L)
            out["dv"][here] = torch.matmul(p.transpose(1, 2), do).transpose(0, 1).to(dt)
            ds = p * (torch.matmul(do, v.transpose(1, 2)) - (do * y).sum(-1, keepdim=True)) * s["scale"]
            out["dq"][here] = _rows(torch.matmul(ds, kk), Hkv, L).to(dt)
            out["dk"][here] = torch.matmul(ds.transpose(1, 2), qg).transpose(0, 1).to(dt)
    return out


# ---- the cache in plain operations ------------------------------------------------------------------------------------


def _places(s, lens, first):
    """For each packed row its page, the block there and the place in the block; and whether that is before `first`."""
    seq, t = _owner(lens)
    t = t + torch.tensor(first, device=DEV)[seq]
    P = s["kc"].shape[2]
    return s["table"].long()[seq, t // P], t % P // BLOCK, t % BLOCK, seq, t


def _quantised(x, scale, old):
    """Codes and scales of blocks x [.., 32, d], at least `old`."""
    most = torch.where(x.isfinite(), x.abs(), 0).amax((-1, -2))
    m, e = torch.frexp(most)  # most = m 2^e with 0.5 <= m < 1; 448 = 0.875 2^9
    need = torch.ldexp(torch.ones_like(m), (e - 9 + (m > 0.875).int()).clamp(min=-117))
    new = torch.maximum(torch.where(most > 0, need, LEAST), torch.where(old, scale, LEAST))
    y = x / new[..., None, None]
    return torch.where(y.isfinite(), y, float("nan")).to(E4M3), new


def _plain_write(s, k, v, lens, first):
    page, blk, off, seq, t = _places(s, lens, first)
    pages, Hkv, P, d = s["kc"].shape
    some, slot = torch.unique(page * (P // BLOCK) + blk, return_inverse=True)
    begin = torch.tensor(first, device=DEV)[seq]
    # how many places at the front of a block hold older tokens
    keep = torch.zeros_like(some)
    front = t // BLOCK == begin // BLOCK
    keep[slot[front]] = (begin % BLOCK)[front]
    older = torch.arange(BLOCK, device=DEV) < keep[:, None]
    live = older.clone()
    live[slot, off] = True  # what stands behind the last token stays
    pg, bl = some // (P // BLOCK), some % (P // BLOCK)
    for x, codes, scales in ((k, s["kc"], s["ks"]), (v, s["vc"], s["vs"])):
        blocks = codes.view(pages, Hkv, P // BLOCK, BLOCK, d)
        sc = scales[pg, :, bl]
        raw = blocks.view(torch.uint8)[pg, :, bl]
        was = raw.view(E4M3).float() * sc[..., None, None]
        now = torch.where(older[:, None, :, None], was, 0)
        now[slot, :, off] = x.float()
        c, sc = _quantised(now, sc, (keep > 0)[:, None])
        blocks.view(torch.uint8)[pg, :, bl] = torch.where(live[:, None, :, None], c.view(torch.uint8), raw)
        scales[pg, :, bl] = sc


def _plain_read(s):
    page, blk, off, _, _ = _places(s, s["new"], s["old"])
    P, dt = s["kc"].shape[2], DT[s["case"]["t"]]
    got = []
    for codes, scales in ((s["kc"], s["ks"]), (s["vc"], s["vs"])):
        x = codes.view(torch.uint8)[page, :, blk * BLOCK + off].view(E4M3).float()
        got.append((x * scales[page, :, blk][..., None]).to(dt))
    return {"k": got[0], "v": got[1]}


def _held(s, codes, scales):
    """[N, longest, Hkv, d]: the cached tokens of every sequence, 0 behind its last."""
    P, longest = codes.shape[2], max(s["whole"])
    t = torch.arange(longest, device=DEV)
    page = s["table"].long()[:, t // P].clamp(min=0)
    x = codes.view(torch.uint8)[page, :, t % P].view(E4M3).float()
    x = x * scales[page, :, t % P // BLOCK][..., None]
    return torch.where((t < s["len"][:, None])[..., None, None], x, 0)


def _plain_decode(s):
    q, (pages, Hkv, P, d) = s["q"], s["kc"].shape
    n, Q = len(s["new"]), max(s["new"])
    seq, i = _owner(s["new"])
    qp = torch.zeros(n, Q, Hkv, q.shape[1] // Hkv, d, device=DEV)
    qp[seq, i] = q.float().unflatten(1, (Hkv, -1))
    qp = qp.permute(0, 2, 1, 3, 4).reshape(n, Hkv, -1, d)  # rows: token, then head of the group
    k = _held(s, s["kc"], s["ks"])
    x = torch.matmul(qp, k.permute(0, 2, 3, 1).contiguous()).view(n, Hkv, Q, -1, k.shape[1]) * s["scale"]
    del k
    last = s["start"][:, None] + torch.arange(Q, device=DEV)
    seen = torch.arange(x.shape[-1], device=DEV) <= last[..., None]
    x = torch.where(seen[:, None, :, None], x, float("-inf"))
    e = torch.exp(x - x.amax(-1, keepdim=True))
    z = e.sum(-1, keepdim=True)
    v = _held(s, s["vc"], s["vs"]).transpose(1, 2).contiguous()
    y = torch.matmul(e.view(n, Hkv, -1, x.shape[-1]), v).view(n, Hkv, Q, -1, d) / z
    return {"o": y.permute(0, 2, 1, 3, 4).flatten(2, 3)[seq, i].to(q.dtype)}


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        from linear_attention_rnn_gated_amd import binding as lib
        if op in ("attn", "train"):
            o, lse = lib.gdn_attn_prefill(s["shape"], s["q"], s["k"], s["v"], s["cu"])
            out = {"o": o, "lse": lse}
            if op == "train":
                out.update(lib.gdn_attn_bwd(s["shape"], s["q"], s["k"], s["v"], s["cu"], o, lse, s["do"], ws=s["ws"]))
            return out
        many = {} if s["one"] else {"cu_seqlens": s["cu"]}
        if op == "write":
            lib.gdn_kv_write(s["shape"], s["k"], s["v"], s["cache"], s["table"], start=s["start"], **many)
            return {"k": s["kc"], "k_scale": s["ks"], "v": s["vc"], "v_scale": s["vs"]}
        if op == "read":
            k, v = lib.gdn_kv_read(s["shape"], s["cache"], s["table"], s["cu"], sum(s["new"]), start=s["start"])
            return {"k": k, "v": v}
        return {"o": lib.gdn_attn_decode(s["shape"], s["q"], s["cache"], s["table"], s["len"], max(s["whole"]), ws=s["ws"],
                                         **many)}
    if op in ("attn", "train"):
        return _plain_attn(s)
    if op == "write":
        _plain_write(s, s["k"], s["v"], s["new"], s["old"])
        return {"k": s["kc"], "k_scale": s["ks"], "v": s["vc"], "v_scale": s["vs"]}
    return _plain_read(s) if op == "read" else _plain_decode(s)


def work(case):
    """Each input read once and each output written once; 2 operations for each product and sum, pairs under the diagonal."""
    size, Hq, Hkv, d = {"f32": 4, "bf16": 2}[case["t"]], case["Hq"], case["Hkv"], case["d"]
    if case["op"] in ("attn", "train"):
        lens = _lens(case["lens"])
        T, pairs = sum(lens), sum(v * (v + 1) // 2 for v in lens)
        rows = T * d * size
        if case["op"] == "attn":
            return {"bytes": rows * (2 * Hq + 2 * Hkv) + T * Hq * 4, "flops": 4 * pairs * Hq * d}
        # forward, then five products more; o and its gradient read, dq, dk and dv written
        return {"bytes": rows * (4 * Hq + 4 * Hkv) + T * Hq * 4, "flops": 14 * pairs * Hq * d}
    old, new = _lens(case["old"], 5), _lens(case["new"])
    T = sum(new)
    if case["op"] in ("write", "read"):
        n = 2 * T * Hkv * d
        return {"bytes": n * (size + 1) + 2 * Hkv * 4 * -(-T // BLOCK), "flops": 2 * n}
    held = sum(old) + T
    pairs = sum(b * a + b * (b + 1) // 2 for a, b in zip(old, new))
    return {"bytes": 2 * held * Hkv * (d + 4 / BLOCK) + 2 * T * Hq * d * size, "flops": 4 * pairs * Hq * d}


# ---- the definitions in 64 bits ---------------------------------------------------------------------------------------


def _exact_attn(case, s):
    """One head at a time; the gradient by differentiating the formula."""
    f64 = dict(dtype=torch.float64, device=DEV)
    T, Hkv, d = s["k"].shape
    G, train = s["q"].shape[1] // Hkv, "do" in s
    out = {"o": torch.zeros(T, Hkv * G, d, **f64), "lse": torch.zeros(T, Hkv * G, **f64)}
    if train:
        out.update(dq=torch.zeros(T, Hkv * G, d, **f64), dk=torch.zeros(T, Hkv, d, **f64), dv=torch.zeros(T, Hkv, d, **f64))
    for a, b in zip(s["cu"].tolist()[:-1], s["cu"].tolist()[1:]):
        above = torch.ones(b - a, b - a, dtype=torch.bool, device=DEV).triu(1)
        for h in range(Hkv * G if b > a else 0):
            q, k, v = (x[a:b, i].double().requires_grad_(train) for x, i in ((s["q"], h), (s["k"], h // G), (s["v"], h // G)))
            x = (q @ k.t() / math.sqrt(d)).masked_fill(above, float("-inf"))
            lse = torch.logsumexp(x, 1)
            o = torch.exp(x - lse[:, None]) @ v
            out["o"][a:b, h], out["lse"][a:b, h] = o.detach(), lse.detach()
            if train:
                g = torch.autograd.grad(o, [q, k, v], s["do"][a:b, h].double())
                out["dq"][a:b, h] = g[0]
                out["dk"][a:b, h // G] += g[1]
                out["dv"][a:b, h // G] += g[2]
    return out


def _values(s, name, n, count):
    """The first `count` cached tokens of sequence n in 64 bits, [count, Hkv, d], page by page."""
    codes, scales, P = s[name + "c"], s[name + "s"], s["kc"].shape[2]
    ids = s["table"][n, :-(-count // P)].tolist()
    x = torch.cat([codes[i].double().unflatten(1, (-1, BLOCK)).mul(scales[i].double()[..., None, None]).flatten(1, 2)
                   .transpose(0, 1) for i in ids])
    return x[:count]


def _exact_write(s):
    """The pool after the write, with x / s before its rounding in the place of the written codes."""
    out, P = {}, s["kc"].shape[2]
    for name in "kv":
        pool, scale = s[name + "c"].double().unflatten(2, (-1, BLOCK)), s[name + "s"].double().clone()
        at = 0
        for n, (a, b) in enumerate(zip(s["old"], s["new"])):
            first = a // BLOCK * BLOCK  # the blocks from here on change
            was = _values(s, name, n, a)[first:] if a else s[name][:0].double()
            x = torch.cat([was, s[name][at:at + b].double()])
            at += b
            count = len(x)
            x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, -count % BLOCK)).unflatten(0, (-1, BLOCK)).permute(0, 2, 1, 3)
            need = torch.exp2(torch.ceil(torch.log2(x.abs().amax((2, 3)) / 448)).clamp(min=-117))
            blk = torch.arange(first // BLOCK, first // BLOCK + len(x), device=DEV)
            page, slot = s["table"][n].long()[blk * BLOCK // P], blk % (P // BLOCK)
            if a > first:
                need[0] = torch.maximum(need[0], scale[page[0], :, slot[0]])
            scale[page, :, slot] = need
            there = (torch.arange(len(x) * BLOCK, device=DEV) < count).view(-1, 1, BLOCK, 1)
            pool[page, :, slot] = torch.where(there, x / need[..., None, None], pool[page, :, slot])
        out[name], out[name + "_scale"] = pool.flatten(2, 3), scale
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("attn", "train"):
        return _exact_attn(case, s)
    if case["op"] == "write":
        return _exact_write(s)
    if case["op"] == "read":
        got = [[_values(s, name, n, a + b)[a:] for n, (a, b) in enumerate(zip(s["old"], s["new"]))] for name in "kv"]
        return {"k": torch.cat(got[0]), "v": torch.cat(got[1])}
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    at, Hkv = 0, case["Hkv"]
    for n, (a, b) in enumerate(zip(s["old"], s["new"])):
        k, v = _values(s, "k", n, a + b), _values(s, "v", n, a + b)
        hidden = torch.ones(b, a + b, dtype=torch.bool, device=DEV).triu(a + 1)
        for h in range(Hkv):
            heads = slice(h * case["Hq"] // Hkv, (h + 1) * case["Hq"] // Hkv)
            q = s["q"][at:at + b, heads].double()
            x = (q.flatten(0, 1) @ k[:, h].t().contiguous()).view(*q.shape[:2], -1) / math.sqrt(case["d"])
            p = torch.softmax(x.masked_fill(hidden[:, None], float("-inf")), -1)
            o[at:at + b, heads] = (p.flatten(0, 1) @ v[:, h]).view(q.shape)
        at += b
    return {"o": o}
