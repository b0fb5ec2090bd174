"""Cases that measure the operators of a linear-attention layer: linear attention with a decay for each
head (packed prompts, training, single tokens) and the pass in front of it that norms the queries and
keys of every head and rotates them to their positions (forward, training).

Sizes come from the packed workloads in linear_attention_chunked_gb300/inputs.py (16384 tokens in
documents of 9000 / 5000 / 2384; 64 or 16 heads of 128 channels) and from generic serving batches.
With ``own`` false every operator is computed by elementary torch operations in 32 bits (the
rotation's angles in 64); with ``own`` true by the library's entry points.
"""
import math
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
D = 128  # head dim of the linear attention


def listed():
    return [
        # a short question to a small model: latency
        dict(name="lin_prompt_short", op="lin_prompt", lens="37", H=8, Hk=8, h0=False),
        # prefill of packed prompts, 64 heads
        dict(name="lin_prompt_3doc", op="lin_prompt", lens="9000,5000,2384", H=64, Hk=64, h0=False),
        # a training step's attention, forward and backward, one long document, 16 heads
        dict(name="lin_train_1doc", op="lin_train", lens="16384", H=16, Hk=16, h0=False),
        # a ragged pack that continues earlier fragments: odd lengths, an empty document, queries and keys shared by three heads
        dict(name="lin_train_ragged", op="lin_train", lens="1,0,777,127,128,129,300", H=6, Hk=2, h0=True),
        # decoding for one user, and for a full serving batch
        dict(name="lin_step_1", op="lin_step", N=1, H=16, Hk=16),
        dict(name="lin_step_256", op="lin_step", N=256, H=64, Hk=64),
        # one decoded token, and a batch of them far into their sequences, four of whose heads share a key head
        dict(name="rope_token", op="rope_fwd", T=1, Hq=16, Hk=16, D=128, R=128, dtype="bf16", norm=True, inter=False, scaling="none", far=100000, fused=True),
        dict(name="rope_tokens_512", op="rope_fwd", T=512, Hq=64, Hk=16, D=128, R=128, dtype="bf16", norm=True, inter=False, scaling="ramp", far=1000000, fused=True),
        # prefill: rotation alone, of half of each head, neighbouring pairs, positions scaled to a longer context
        dict(name="rope_prompt_part", op="rope_fwd", T=16384, Hq=64, Hk=64, D=128, R=64, dtype="bf16", norm=False, inter=True, scaling="linear", far=0, fused=True),
        # a training step, norm and rotation, forward and backward
        dict(name="rope_train_16k", op="rope_train", T=16384, Hq=64, Hk=64, D=128, R=128, dtype="bf16", norm=True, inter=False, scaling="none", far=0, fused=True),
        # odd sizes in 32 bits
        dict(name="rope_train_ragged", op="rope_train", T=1777, Hq=7, Hk=3, D=80, R=52, dtype="fp32", norm=True, inter=False, scaling="base", far=0, fused=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lens(rng, total):
    n = min(_log(rng, 1, 12), total)
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [total]))


def draw(rng):
    op = rng.choice(["lin_prompt", "lin_train", "lin_step", "rope_fwd", "rope_train"])
    if op.startswith("lin"):
        Hk = _log(rng, 1, 64)
        share = rng.choice([1, 1, 1, 2, 3, 4])
        H = min(Hk * share, 64) // Hk * Hk
        if op == "lin_step":
            return dict(op=op, N=_log(rng, 1, 256), H=H, Hk=Hk)
        room = 16384 * (64 if op == "lin_prompt" else 16) // H
        return dict(op=op, lens=_lens(rng, _log(rng, 16, min(16384, room))), H=H, Hk=Hk, h0=rng.random() < 0.5)
    dim = rng.choice([128, 128, 64, 256, 80, 96, 2 * rng.randint(8, 128)])
    R = rng.choice([dim, dim, 2 * rng.randint(1, dim // 2), 8 * rng.randint(1, dim // 8)])
    Hq, Hk = _log(rng, 1, 64), _log(rng, 1, 64)
    T = _log(rng, 1, min(16384, 16384 * 128 * 128 // ((Hq + Hk) * dim) // (1 if op == "rope_train" else 1)))
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if dtype == "fp32":
        T = max(1, T // 2)
    return dict(op=op, T=T, Hq=Hq, Hk=Hk, D=dim, R=R, dtype=dtype, norm=rng.random() < 0.6, inter=rng.random() < 0.5,
                scaling=rng.choice(["none", "linear", "base", "ramp"]), far=rng.choice([0, 1000, 100000, 1000000]),
                fused=rng.random() < 0.5)


def _cu(case):
    out = [0]
    for n in case["lens"].split(","):
        out.append(out[-1] + int(n))
    return out


def _frequencies(R, scaling):
    """Radians per token of the R / 2 pairs, and the factor on the rotated values."""
    base, factor, trained = 10000.0, 8.0, 4096
    if scaling == "base":
        base *= factor ** (R / max(R - 2, 1))
    f = [base ** (-2.0 * i / R) for i in range(R // 2)]
    if scaling == "linear":
        return [x / factor for x in f], 1.0
    if scaling == "ramp":  # pairs that turn rarely within the trained length are stretched, the others kept
        out = []
        for x in f:
            turns = trained * x / (2 * math.pi)
            keep = min(max((turns - 1.0) / (32.0 - 1.0), 0.0), 1.0)
            out.append(x * keep + x / factor * (1.0 - keep))
        return out, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    st = dict(case)
    op = case["op"]
    if op.startswith("lin"):
        H, Hk = case["H"], case["Hk"]
        if op == "lin_step":
            rows = docs = case["N"]
        else:
            st["cu_host"] = _cu(case)
            rows, docs = st["cu_host"][-1], len(st["cu_host"]) - 1
            st["cu"] = torch.tensor(st["cu_host"], dtype=torch.int32, device="cuda")
        # queries, keys and values are columns of one projection
        qkv = randn(rows, (2 * Hk + H) * D).bfloat16()
        st["q"] = qkv[:, :Hk * D].unflatten(1, (Hk, D))
        st["k"] = qkv[:, Hk * D:2 * Hk * D].unflatten(1, (Hk, D))
        st["v"] = qkv[:, 2 * Hk * D:].unflatten(1, (H, D))
        # log decays from about -0.9 (a few tokens) to -1/256 (some hundred), a geometric row over the heads
        at = (torch.arange(H, device="cuda") + torch.rand((H,), generator=gen, device="cuda")) / H
        st["slope"] = -torch.exp2(-8.0 * at)
        st["scale"] = D ** -0.5
        if op == "lin_step":
            st["h"] = randn(docs, H, D, D)
            st["h_out"] = torch.empty_like(st["h"])
        else:
            st["h0"] = randn(docs, H, D, D) if case["h0"] else None
        if op == "lin_train":
            st["do"] = randn(rows, H, D).bfloat16()
            st["dht"] = 0.1 * randn(docs, H, D, D) if case["h0"] else None
        return st
    T, Hq, Hk, dim, dt = case["T"], case["Hq"], case["Hk"], case["D"], _DT[case["dtype"]]
    if case["fused"]:  # columns of one projection that also holds the values
        qkv = (1.5 * randn(T, (Hq + 2 * Hk) * dim)).to(dt)
        st["q"] = qkv[:, :Hq * dim].unflatten(1, (Hq, dim))
        st["k"] = qkv[:, Hq * dim:(Hq + Hk) * dim].unflatten(1, (Hk, dim))
    else:
        st["q"], st["k"] = (1.5 * randn(T, Hq, dim)).to(dt), (1.5 * randn(T, Hk, dim)).to(dt)
    f, st["factor"] = _frequencies(case["R"], case["scaling"])
    st["freq"] = torch.tensor(f, dtype=torch.float64, device="cuda")
    if case["far"]:  # single tokens of sequences of any length
        st["pos"] = torch.randint(0, case["far"] + 1, (T,), generator=gen, device="cuda", dtype=torch.int32)
    else:
        st["pos"] = torch.arange(T, device="cuda", dtype=torch.int32)
    st["wq"] = 1.0 + 0.1 * randn(dim) if case["norm"] else None
    st["wk"] = 1.0 + 0.1 * randn(dim) if case["norm"] else None
    if op == "rope_train":
        st["dq"], st["dk"] = randn(T, Hq, dim).to(dt), randn(T, Hk, dim).to(dt)
    return st


def run(st):
    return (_run_own if own else _run_plain)(st)


# ---- the library's entry points ----

def _run_own(st):
    from linear_attention_chunked_gb300 import kda
    op = st["op"]
    if op == "lin_step":
        return kda.kda_linattn_step(st["q"], st["k"], st["v"], st["slope"], st["h"], scale=st["scale"], h_out=st["h_out"])
    if op.startswith("lin"):
        a = (st["q"], st["k"], st["v"], st["slope"], st["cu"])
        kw = dict(h0=st["h0"], scale=st["scale"])
        o, ht, saved = kda.kda_linattn_fwd(*a, **kw, save=op == "lin_train")
        if op == "lin_prompt":
            return o, ht
        g = kda.kda_linattn_bwd(*a, st["do"], **kw, dht=st["dht"], saved=saved, want_dh0=st["h0"] is not None)
        return dict(g, o=o, ht=ht)
    kw = dict(wq=st["wq"], wk=st["wk"], norm=st["norm"], eps=1e-6, interleaved=st["inter"], scale=st["factor"])
    q, k = kda.kda_rope_fwd(st["q"], st["k"], st["pos"], st["freq"], **kw)
    out = dict(q=q, k=k)
    if op == "rope_train":
        out.update(kda.kda_rope_bwd(st["q"], st["k"], st["pos"], st["freq"], st["dq"], st["dk"], **kw))
    return out


# ---- the plain forms ----

def _shared(x, H):
    """[rows, Hk, D] -> [H, rows, D] in 32 bits, each query or key head repeated for the heads that share it."""
    return x.float().repeat_interleave(H // x.shape[1], dim=1).transpose(0, 1)


def _plain_lin(st):
    H, Hk, slope, scale = st["H"], st["Hk"], st["slope"], st["scale"]
    train = st["op"] == "lin_train"
    q, k, v = _shared(st["q"], H), _shared(st["k"], H), _shared(st["v"], H)
    cu, C, dev = st["cu_host"], 128, st["q"].device
    n = torch.arange(C + 1, device=dev)
    power = torch.exp(slope[:, None] * n)[:, :, None]
    gap = n[:C, None] - n[None, :C]
    mask = torch.where(gap >= 0, torch.exp(slope[:, None, None] * gap.clamp(min=0)), 0.0)
    N = len(cu) - 1
    o = torch.empty_like(v)
    ht = torch.zeros((N, H, D, D), device=dev)
    if train:
        do = _shared(st["do"], H)
        dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(v)
        dh0 = torch.zeros_like(ht)
    for i in range(N):
        S = st["h0"][i] if st["h0"] is not None else ht[i]
        starts = range(cu[i], cu[i + 1], C)
        for c in starts:
            e = min(c + C, cu[i + 1])
            m = e - c
            qc, kc, vc = q[:, c:e], k[:, c:e], v[:, c:e]
            M = mask[:, :m, :m]
            o[:, c:e] = scale * (((qc @ kc.transpose(1, 2)) * M) @ vc + power[:, 1:m + 1] * (qc @ S))
            if train:
                doc = scale * do[:, c:e]
                dq[:, c:e] = ((doc @ vc.transpose(1, 2)) * M) @ kc + power[:, 1:m + 1] * (doc @ S.transpose(1, 2))
            S = power[:, m, :, None] * S + (kc * power[:, :m].flip(1)).transpose(1, 2) @ vc
        ht[i] = S
        if not train:
            continue
        G = st["dht"][i] if st["dht"] is not None else dh0[i]
        for c in reversed(starts):
            e = min(c + C, cu[i + 1])
            m = e - c
            qc, kc, vc, doc = q[:, c:e], k[:, c:e], v[:, c:e], scale * do[:, c:e]
            M = mask[:, :m, :m]
            back = power[:, :m].flip(1)
            dv[:, c:e] = ((qc @ kc.transpose(1, 2)) * M).transpose(1, 2) @ doc + back * (kc @ G)
            dk[:, c:e] = ((doc @ vc.transpose(1, 2)) * M).transpose(1, 2) @ qc + back * (vc @ G.transpose(1, 2))
            G = power[:, m, :, None] * G + (qc * power[:, 1:m + 1]).transpose(1, 2) @ doc
        dh0[i] = G
    rows = lambda x: x.transpose(0, 1).to(torch.bfloat16)  # noqa: E731
    if not train:
        return rows(o).contiguous(), ht
    group = lambda x: x.unflatten(0, (Hk, H // Hk)).sum(1)  # noqa: E731
    out = dict(o=rows(o).contiguous(), ht=ht, dq=rows(group(dq)).contiguous(), dk=rows(group(dk)).contiguous(),
               dv=rows(dv).contiguous())
    if st["h0"] is not None:
        out["dh0"] = dh0
    return out


def _parts(x, R, inter):
    """The two members of every rotated pair, and the rest of the head."""
    if inter:
        return x[..., 0:R:2], x[..., 1:R:2], x[..., R:]
    return x[..., :R // 2], x[..., R // 2:R], x[..., R:]


def _joined(a, b, rest, inter):
    turned = torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)
    return torch.cat([turned, rest], -1)


def _plain_rope(st, x, w, dy):
    f, R, inter = torch.float32, st["R"], st["inter"]
    angle = st["pos"].double()[:, None, None] * st["freq"]
    cos, sin = (torch.cos(angle) * st["factor"]).to(f), (torch.sin(angle) * st["factor"]).to(f)
    v = x.to(f)
    if st["norm"]:
        r = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6)
        xh = v * r
        v = xh * w
    if dy is None:
        a, b, rest = _parts(v, R, inter)
        return _joined(a * cos - b * sin, a * sin + b * cos, rest, inter).to(x.dtype)
    a, b, rest = _parts(dy.to(f), R, inter)
    d = _joined(a * cos + b * sin, b * cos - a * sin, rest, inter)
    if not st["norm"]:
        return d.to(x.dtype), None
    dw = (d * xh).sum((0, 1))
    d = d * w
    return (r * (d - xh * (d * xh).mean(-1, keepdim=True))).to(x.dtype), dw


def _run_plain(st):
    op = st["op"]
    if op == "lin_step":
        H = st["H"]
        q, k, v = (_shared(st[n], H).transpose(0, 1) for n in "qkv")
        h = torch.exp(st["slope"])[:, None, None] * st["h"] + k[..., None] * v[..., None, :]
        return (st["scale"] * (q[..., None] * h).sum(2)).bfloat16(), h
    if op.startswith("lin"):
        return _plain_lin(st)
    out = dict(q=_plain_rope(st, st["q"], st["wq"], None), k=_plain_rope(st, st["k"], st["wk"], None))
    if op == "rope_train":
        out["dq"], dwq = _plain_rope(st, st["q"], st["wq"], st["dq"])
        out["dk"], dwk = _plain_rope(st, st["k"], st["wk"], st["dk"])
        if st["norm"]:
            out["dwq"], out["dwk"] = dwq, dwk
    return out


# ---- the definitions in 64 bits ----

def exact(case, seed):
    st = prepare(case, seed)
    d, op = torch.float64, case["op"]
    v = {key: (x.to(d) if torch.is_tensor(x) and x.is_floating_point() else x) for key, x in st.items()}
    if op == "lin_step":
        share = case["H"] // case["Hk"]
        heads = torch.arange(case["H"], device="cuda") // share
        o, h = [], []
        for n in range(case["N"]):  # one sequence after the other
            state = v["h"][n] * torch.exp(v["slope"]).view(-1, 1, 1)
            state += torch.einsum("hi,hj->hij", v["k"][n, heads], v["v"][n])
            o.append(v["scale"] * torch.einsum("hi,hij->hj", v["q"][n, heads], state))
            h.append(state)
        return torch.stack(o), torch.stack(h)
    if op.startswith("lin"):
        return _exact_lin(case, v)

    def turn(x, w, back):
        """Pairs as complex numbers, turned by their angles."""
        T, R = case["T"], case["R"]
        if back is None and case["norm"]:
            x = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + 1e-6) * w
        src = x if back is None else back
        z = src[..., :R].unflatten(-1, (-1, 2)) if case["inter"] else src[..., :R].unflatten(-1, (2, -1)).transpose(-1, -2)
        c = torch.view_as_complex(z.contiguous())
        angle = (v["pos"].to(d).view(T, 1, 1) * v["freq"]) * (1 if back is None else -1)
        z = torch.view_as_real(c * torch.polar(torch.full_like(angle, v["factor"]), angle))
        z = z.flatten(-2) if case["inter"] else z.transpose(-1, -2).flatten(-2)
        return torch.cat([z, src[..., R:]], -1)

    out = dict(q=turn(v["q"], v["wq"], None), k=turn(v["k"], v["wk"], None))
    if op == "rope_train":
        for name in "qk":
            x, w, g = v[name], v["w" + name], turn(v[name], v["w" + name], v["d" + name])
            if case["norm"]:
                s = x.pow(2).mean(-1, keepdim=True) + 1e-6
                out["dw" + name] = (g * x / s.sqrt()).sum((0, 1))
                g = g * w
                g = g / s.sqrt() - x * (g * x).mean(-1, keepdim=True) / s.pow(1.5)
            out["d" + name] = g
    return out


def _exact_lin(case, v):
    """Every pair of tokens of a document at once, head by head."""
    H, share, cu, scale = case["H"], case["H"] // case["Hk"], v["cu_host"], v["scale"]
    train = case["op"] == "lin_train"
    lens = [b - a for a, b in zip(cu, cu[1:])]
    if sum(n * n for n in lens) * H * D * 4 * (3 if train else 1) > 1.2e13:
        return None
    T, N = cu[-1], len(lens)
    o = torch.zeros_like(v["v"])
    ht = torch.zeros((N, H, D, D), dtype=torch.float64, device="cuda")
    dq, dk = torch.zeros_like(v["q"]), torch.zeros_like(v["k"])
    dv, dh0 = torch.zeros_like(o), torch.zeros_like(ht)
    for i in range(N):
        r = slice(cu[i], cu[i + 1])
        at = torch.arange(lens[i], device="cuda", dtype=torch.float64)
        for h in range(H):
            a = v["slope"][h]
            q, k, x = v["q"][r, h // share], v["k"][r, h // share], v["v"][r, h]
            W = torch.exp(a * (at[:, None] - at)).tril_()
            start = torch.exp(a * (at + 1))[:, None]
            end = torch.exp(a * (lens[i] - 1 - at))[:, None]
            kv0 = v["h0"][i, h] if v["h0"] is not None else None
            o[r, h] = scale * ((q @ k.T) * W) @ x
            ht[i, h] = (k * end).T @ x
            if kv0 is not None:
                o[r, h] += scale * start * (q @ kv0)
                ht[i, h] += torch.exp(a * lens[i]) * kv0
            if not train:
                continue
            g = scale * v["do"][r, h]
            dA = (g @ x.T) * W
            dq[r, h // share] += dA @ k
            dk[r, h // share] += dA.T @ q
            dv[r, h] = ((q @ k.T) * W).T @ g
            if kv0 is not None:
                G = v["dht"][i, h]
                dq[r, h // share] += start * (g @ kv0.T)
                dk[r, h // share] += end * (x @ G.T)
                dv[r, h] += end * (k @ G)
                dh0[i, h] = torch.exp(a * lens[i]) * G + (q * start).T @ g
    if not train:
        return o, ht
    out = dict(o=o, ht=ht, dq=dq, dk=dk, dv=dv)
    if v["h0"] is not None:
        out["dh0"] = dh0
    return out


def work(case):
    op = case["op"]
    if op.startswith("lin"):
        H, Hk = case["H"], case["Hk"]
        lens = [int(n) for n in case["lens"].split(",")] if "lens" in case else [1] * case["N"]
        T, N, state = sum(lens), len(lens), 4 * H * D * D
        rows = 2 * T * D * (2 * Hk + 2 * H) + 4 * H
        if op == "lin_step":
            return {"bytes": rows + 2 * N * state, "flops": 5 * T * H * D * D}
        data, flops = rows + N * state * (2 if case["h0"] else 1), 5 * T * H * D * D
        if op == "lin_train":
            data += 2 * T * D * (2 * Hk + 2 * H) + (2 * N * state if case["h0"] else 0)
            flops += 9 * T * H * D * D
        return {"bytes": data, "flops": flops}
    e, dim = _BYTES[case["dtype"]], case["D"]
    n = case["T"] * (case["Hq"] + case["Hk"]) * dim
    data, flops = 2 * e * n + 4 * case["T"] + 4 * case["R"], n * (7 if case["norm"] else 3)
    if op == "rope_train":
        data, flops = data + 2 * e * n, flops + n * (14 if case["norm"] else 3)
    return {"bytes": data, "flops": flops}
