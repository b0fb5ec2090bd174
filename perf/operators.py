"""Cases that measure the state-space block's operators: the selective scan (prompts, training,
single tokens), its short causal conv in serving (prompt with the window it leaves, single
tokens) and the layer norm (forward, training).

Sizes come from the packed workloads in linear_attention_chunked_gb300/inputs.py (16384 tokens in
documents of 8192 / 4096 / 3072 / 1024 or 9000 / 5000 / 2384; 64 or 16 heads of 128 channels) and
from generic serving batches.  With ``own`` false every operator is computed by elementary torch
operations in 32 bits; with ``own`` true by the library's entry points.
"""
import math
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # a short question to a small model: latency
        dict(name="scan_prompt_short", op="scan_prompt", lens="37", C=1024, S=16, G=1, dtype="bf16", z=True, h0=False),
        # prefill of packed prompts at the width of 64 heads x 128 channels
        dict(name="scan_prompt_4doc", op="scan_prompt", lens="8192,4096,3072,1024", C=8192, S=16, G=1, dtype="bf16", z=True, h0=False),
        # a training step's scan, forward and backward, 16 heads x 128 channels
        dict(name="scan_train_4doc", op="scan_train", lens="8192,4096,3072,1024", C=2048, S=16, G=1, dtype="bf16", z=True, h0=False),
        # ragged pack that continues earlier fragments: odd lengths, an empty document, two groups, fp32
        dict(name="scan_train_ragged", op="scan_train", lens="1,0,777,63,64,65,300", C=392, S=12, G=2, dtype="fp32", z=False, h0=True),
        # decoding for one user, and for a full serving batch
        dict(name="scan_step_1", op="scan_step", N=1, C=2048, S=16, G=1, dtype="bf16", z=True),
        dict(name="scan_step_256", op="scan_step", N=256, C=8192, S=16, G=1, dtype="bf16", z=True),
        # the conv ahead of the scan: packed prompts with the window they leave; single tokens
        dict(name="conv_prompt_3doc", op="conv_prompt", lens="9000,5000,2384", C=2048, halo=False),
        dict(name="conv_step_1", op="conv_step", N=1, C=2048),
        dict(name="conv_step_512", op="conv_step", N=512, C=8192),
        # the norm in front of a block: one decoded token per sequence with its residual; a training step; odd sizes
        dict(name="norm_token", op="norm_fwd", T=8, C=2048, dtype="bf16", res=True),
        dict(name="norm_train_16k", op="norm_train", T=16384, C=8192, dtype="bf16", res=False),
        dict(name="norm_train_ragged", op="norm_train", T=1777, C=1111, dtype="fp32", res=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lens(rng, total):
    n = min(_log(rng, 1, 12), total)
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [total]))


def draw(rng):
    op = rng.choice(["scan_prompt", "scan_train", "scan_step", "conv_prompt", "conv_step", "norm_fwd", "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("scan_prompt", "scan_train", "scan_step"):
        G = rng.choice([1, 1, 1, 2, 4])
        C = G * max(1, _log(rng, 256, 8192 if op != "scan_train" else 2048) // G)
        S = rng.choice([16, 16, 16, 4, 8, 12, 32, 64])
        room = 16384 * 2048 * 16 // (C * S)
        if op == "scan_step":
            return dict(op=op, N=_log(rng, 1, min(512, room)), C=C, S=S, G=G, dtype=dtype, z=rng.random() < 0.7)
        return dict(op=op, lens=_lens(rng, _log(rng, 16, max(17, min(16384, room)))), C=C, S=S, G=G, dtype=dtype,
                    z=rng.random() < 0.7, h0=rng.random() < 0.5)
    if op == "conv_prompt":
        return dict(op=op, lens=_lens(rng, _log(rng, 16, 16384)), C=8 * _log(rng, 8, 512), halo=rng.random() < 0.5)
    if op == "conv_step":
        return dict(op=op, N=_log(rng, 1, 512), C=8 * _log(rng, 8, 1024))
    C = _log(rng, 64, 16384)
    return dict(op=op, T=_log(rng, 1, min(32768, 16384 * 8192 // C)), C=C, dtype=dtype, res=rng.random() < 0.5)


def _cu(case):
    out = [0]
    for n in case["lens"].split(","):
        out.append(out[-1] + int(n))
    return out


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    st = dict(case)
    op = case["op"]
    C = case["C"]
    if op.startswith("scan"):
        dt, S, G = _DT[case["dtype"]], case["S"], case["G"]
        if op == "scan_step":
            rows, docs = case["N"], case["N"]
        else:
            st["cu_host"] = _cu(case)
            rows, docs = st["cu_host"][-1], len(st["cu_host"]) - 1
            st["cu"] = torch.tensor(st["cu_host"], dtype=torch.int32, device="cuda")
        st["u"] = randn(rows, C).to(dt)
        # delta = softplus(dt + bias) around 0.001 .. 0.1 per channel, as state-space layers start out
        delta = torch.exp(torch.rand((C,), generator=gen, device="cuda") * math.log(100.0) + math.log(1e-3))
        st["dt_bias"] = delta + torch.log(-torch.expm1(-delta))
        st["dt"] = (0.5 * randn(rows, C)).to(dt)
        st["A"] = -(1.0 + torch.arange(S, device="cuda")) * torch.exp(0.2 * randn(C, S))
        st["D"] = 1.0 + 0.1 * randn(C)
        # B and C are columns of one projection, z the second half of another: row-strided views
        proj = randn(rows, 2 * G * S).to(dt)
        st["B"], st["Cm"] = proj[:, :G * S].unflatten(1, (G, S)), proj[:, G * S:].unflatten(1, (G, S))
        st["z"] = randn(rows, 2 * C).to(dt)[:, C:] if case["z"] else None
        if op == "scan_step":
            st["h"] = randn(docs, C, S)
            st["h_out"] = torch.empty_like(st["h"])
        else:
            st["h0"] = randn(docs, C, S) if case["h0"] else None
        if op == "scan_train":
            st["dy"] = randn(rows, C).to(dt)
            st["dht"] = 0.1 * randn(docs, C, S) if case["h0"] else None
    elif op.startswith("conv"):
        st["w"], st["bias"] = 0.5 * randn(C, 4), 0.1 * randn(C)
        if op == "conv_prompt":
            st["cu_host"] = _cu(case)
            st["cu"] = torch.tensor(st["cu_host"], dtype=torch.int32, device="cuda")
            st["x"] = randn(st["cu_host"][-1], C).bfloat16()
            st["halo"] = randn(len(st["cu_host"]) - 1, 3, C).bfloat16() if case["halo"] else None
        else:
            st["x"], st["win"] = randn(case["N"], C).bfloat16(), randn(case["N"], 3, C).bfloat16()
            st["win_out"] = torch.empty_like(st["win"])
    else:
        dt, T = _DT[case["dtype"]], case["T"]
        st["x"] = (2.0 * randn(T, C) + 0.5).to(dt)
        st["resid"] = randn(T, C).to(dt) if case["res"] else None
        st["w"], st["b"] = 1.0 + 0.1 * randn(C), 0.1 * randn(C)
        if op == "norm_train":
            st["dy"] = randn(T, C).to(dt)
            st["dsum"] = randn(T, C).to(dt) if case["res"] else None
    return st


def run(st):
    return (_run_own if own else _run_plain)(st)


# ---- the library's entry points ----

def _run_own(st):
    from linear_attention_chunked_gb300 import kda
    op = st["op"]
    if op == "scan_step":
        return kda.kda_ssm_step(st["u"], st["dt"], st["A"], st["B"], st["Cm"], st["h"], D=st["D"], dt_bias=st["dt_bias"],
                                z=st["z"], h_out=st["h_out"])
    if op.startswith("scan"):
        a = (st["u"], st["dt"], st["A"], st["B"], st["Cm"], st["cu"])
        kw = dict(D=st["D"], dt_bias=st["dt_bias"], z=st["z"], h0=st["h0"])
        y, ht, saved = kda.kda_ssm_fwd(*a, **kw, save=op == "scan_train")
        if op == "scan_prompt":
            return y, ht
        g = kda.kda_ssm_bwd(*a, st["dy"], **kw, dht=st["dht"], saved=saved, want_dh0=st["h0"] is not None)
        return dict(g, y=y, ht=ht)
    if op == "conv_prompt":
        y = kda.kda_conv_fwd(st["x"], st["w"], st["cu"], bias=st["bias"], halo=st["halo"])
        return y, kda.kda_conv_tail(st["x"], st["cu"], halo=st["halo"])
    if op == "conv_step":
        return kda.kda_conv_step(st["x"], st["w"], st["win"], bias=st["bias"], win_out=st["win_out"])
    y, total, mean, rstd = kda.kda_layernorm_fwd(st["x"], st["w"], st["b"], res=st["resid"])
    out = dict(y=y)
    if st["resid"] is not None:
        out["sum"] = total
    if op == "norm_train":
        out.update(kda.kda_layernorm_bwd(total, st["w"], mean, rstd, st["dy"], dsum=st["dsum"]))
    return out


# ---- the plain forms ----

def _scan(a, b, longest):
    """h_t = a_t h_{t-1} + b_t along the first axis, by doubling; a = 0 where a document starts.  In place."""
    d = 1
    while d < longest:
        b[d:] += a[d:] * b[:-d]
        a[d:] = a[d:] * a[:-d]
        d *= 2
    return b


def _per_channel(x, C):
    """[rows, G, S] -> [rows, C, S] of the groups' values (a view where there is one group)."""
    r, G, S = x.shape
    return x[:, :, None, :].expand(r, G, C // G, S).reshape(r, C, S) if G > 1 else x.expand(r, C, S)


def _plain_scan(st, train):
    f = torch.float32
    u, dt, A, D = st["u"].to(f), st["dt"].to(f) + st["dt_bias"], st["A"], st["D"]
    B, Cm = _per_channel(st["B"].to(f), st["C"]), _per_channel(st["Cm"].to(f), st["C"])
    cu, dev = st["cu_host"], st["u"].device
    full = [n for n in range(len(cu) - 1) if cu[n + 1] > cu[n]]
    longest = max([cu[n + 1] - cu[n] for n in full], default=0)
    docs = torch.tensor(full, device=dev)
    first = torch.tensor([cu[n] for n in full], device=dev)
    last = torch.tensor([cu[n + 1] - 1 for n in full], device=dev)
    delta = torch.clamp(dt, min=0) + torch.log1p(torch.exp(-dt.abs()))
    a = torch.exp(delta[:, :, None] * A)
    h = (delta * u)[:, :, None] * B
    if st["h0"] is not None:
        h[first] += a[first] * st["h0"][docs]
    ht = st["h0"].clone() if st["h0"] is not None else torch.zeros((len(cu) - 1, *A.shape), device=dev)
    a0 = a[first]
    a[first] = 0
    h = _scan(a.clone() if train else a, h, longest)
    ht[docs] = h[last]
    y0 = (h * Cm).sum(-1) + D * u
    z = st["z"].to(f) if st["z"] is not None else None
    sg = 1 / (1 + torch.exp(-z)) if z is not None else None
    y = y0 * (z * sg) if z is not None else y0
    out = dict(y=y.to(st["u"].dtype), ht=ht)
    if not train:
        return out["y"], ht
    dy = st["dy"].to(f)
    if z is not None:
        out["dz"] = (dy * y0 * sg * (1 + z * (1 - sg))).to(st["u"].dtype)
        dy = dy * (z * sg)
    g = dy[:, :, None] * Cm
    if st["dht"] is not None:
        g[last] += st["dht"][docs]
    nxt = torch.zeros_like(a)
    nxt[:-1] = a[1:]  # a of the next token of the same document (a is 0 where a document starts)
    g = _scan(nxt.flip(0), g.flip(0), longest).flip(0)
    del nxt
    T, C, S = g.shape
    G = st["G"]
    out["dC"] = (dy[:, :, None] * h).reshape(T, G, C // G, S).sum(2).to(st["u"].dtype)
    out["dB"] = (g * (delta * u)[:, :, None]).reshape(T, G, C // G, S).sum(2).to(st["u"].dtype)
    sB = (g * B).sum(-1)
    prev = torch.zeros_like(h)
    prev[1:] = h[:-1]
    if st["h0"] is not None:
        prev[first] = st["h0"][docs]
        out["dh0"] = st["dht"].clone()
        out["dh0"][docs] = a0 * g[first]
    else:
        prev[first] = 0
    a[first] = a0
    w = g * a * prev
    ddt = (u * sB + (w * A).sum(-1)) / (1 + torch.exp(-dt))
    out["du"] = (delta * sB + D * dy).to(st["u"].dtype)
    out["ddt"] = ddt.to(st["u"].dtype)
    out["dA"], out["dD"], out["ddt_bias"] = (w * delta[:, :, None]).sum(0), (dy * u).sum(0), ddt.sum(0)
    return out


def _run_plain(st):
    f, op = torch.float32, st["op"]
    if op == "scan_step":
        u, dt = st["u"].to(f), st["dt"].to(f) + st["dt_bias"]
        B, Cm = _per_channel(st["B"].to(f), st["C"]), _per_channel(st["Cm"].to(f), st["C"])
        delta = torch.clamp(dt, min=0) + torch.log1p(torch.exp(-dt.abs()))
        h = torch.exp(delta[:, :, None] * st["A"]) * st["h"] + (delta * u)[:, :, None] * B
        y = (h * Cm).sum(-1) + st["D"] * u
        if st["z"] is not None:
            z = st["z"].to(f)
            y = y * z / (1 + torch.exp(-z))
        return y.to(st["u"].dtype), h
    if op.startswith("scan"):
        return _plain_scan(st, op == "scan_train")
    if op == "conv_prompt":
        cu, T, dev = st["cu_host"], st["x"].shape[0], st["x"].device
        N, C = len(cu) - 1, st["C"]
        # every document with the three rows before it in front: rows cu[n] + 3 n .. of one padded tensor
        lens = torch.tensor([cu[n + 1] - cu[n] for n in range(N)], device=dev)
        doc = torch.repeat_interleave(torch.arange(N, device=dev), lens, output_size=T)
        at = torch.arange(T, device=dev) + 3 * (doc + 1)
        pad = torch.zeros((T + 3 * N, C), dtype=f, device=dev)
        pad[at] = st["x"].to(f)
        head = (st["cu"][:-1].long() + 3 * torch.arange(N, device=dev))[:, None] + torch.arange(3, device=dev)
        if st["halo"] is not None:
            pad[head.reshape(-1)] = st["halo"].to(f).reshape(-1, C)
        v = st["bias"] + st["w"][:, 0] * pad[at - 3] + st["w"][:, 1] * pad[at - 2] + st["w"][:, 2] * pad[at - 1] + st["w"][:, 3] * pad[at]
        tail = pad[(head + lens[:, None]).reshape(-1)].reshape(N, 3, C)
        return (v / (1 + torch.exp(-v))).to(st["x"].dtype), tail.to(st["x"].dtype)
    if op == "conv_step":
        rows = torch.cat([st["win"], st["x"][:, None]], 1)
        v = (rows.to(f) * st["w"].t()).sum(1) + st["bias"]
        return (v / (1 + torch.exp(-v))).to(st["x"].dtype), rows[:, 1:].contiguous()
    v = st["x"].to(f)
    if st["resid"] is not None:
        v = (v + st["resid"].to(f)).to(st["x"].dtype).to(f)  # the sum is handed on in the inputs' type, and normalised as it is
    mean = v.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(((v - mean) ** 2).mean(-1, keepdim=True) + 1e-5)
    xh = (v - mean) * rstd
    out = dict(y=(xh * st["w"] + st["b"]).to(st["x"].dtype))
    if st["resid"] is not None:
        out["sum"] = v.to(st["x"].dtype)
    if op == "norm_train":
        dy = st["dy"].to(f)
        d = dy * st["w"]
        dx = rstd * (d - d.mean(-1, keepdim=True) - xh * (d * xh).mean(-1, keepdim=True))
        if st["dsum"] is not None:
            dx = dx + st["dsum"].to(f)
        out["dx"], out["dw"], out["db"] = dx.to(st["x"].dtype), (dy * xh).sum(0), dy.sum(0)
    return out


# ---- the definitions in 64 bits, token by token ----

def exact(case, seed):
    st = prepare(case, seed)
    d, op = torch.float64, case["op"]
    v = {k: (x.to(d) if torch.is_tensor(x) and x.is_floating_point() else x) for k, x in st.items()}
    if op.startswith("scan"):
        return _exact_scan(case, v)
    if op.startswith("conv"):
        act = lambda q: q * torch.sigmoid(q)  # noqa: E731
        if op == "conv_step":
            q = v["bias"] + v["w"][:, 3] * v["x"] + sum(v["w"][:, j] * v["win"][:, j] for j in range(3))
            return act(q), torch.stack([v["win"][:, 1], v["win"][:, 2], v["x"]], 1)
        ys, tails = [], []
        cu = v["cu_host"]
        for n in range(len(cu) - 1):
            front = v["halo"][n] if v["halo"] is not None else torch.zeros((3, case["C"]), dtype=d, device="cuda")
            p = torch.cat([front, v["x"][cu[n]:cu[n + 1]]])
            L = cu[n + 1] - cu[n]
            ys.append(act(v["bias"] + sum(v["w"][:, j] * p[j:j + L] for j in range(4))))
            tails.append(p[L:])
        return torch.cat(ys), torch.stack(tails)
    x = v["x"]
    if v["resid"] is not None:
        x = (x + v["resid"]).to(torch.float32).to(_DT[case["dtype"]]).to(d)  # as handed on
    var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
    xh = (x - mean) / torch.sqrt(var + 1e-5)
    out = dict(y=xh * v["w"] + v["b"])
    if v["resid"] is not None:
        out["sum"] = x
    if op == "norm_train":
        q = v["dy"] * v["w"]
        dx = (q - q.mean(-1, keepdim=True) - xh * (q * xh).mean(-1, keepdim=True)) / torch.sqrt(var + 1e-5)
        out["dx"] = dx + v["dsum"] if v["dsum"] is not None else dx
        out["dw"], out["db"] = (v["dy"] * xh).sum(0), v["dy"].sum(0)
    return out


def _exact_scan(case, v):
    d, C, S, G = torch.float64, case["C"], case["S"], case["G"]
    group = torch.arange(C, device="cuda") // (C // G)
    raw = v["dt"] + v["dt_bias"]
    delta = torch.logaddexp(raw, torch.zeros_like(raw))
    u, A = v["u"], v["A"]
    gate = v["z"] * torch.sigmoid(v["z"]) if v["z"] is not None else None
    if case["op"] == "scan_step":
        h = torch.exp(delta[..., None] * A) * v["h"] + (delta * u)[..., None] * v["B"][:, group]
        y = (h * v["Cm"][:, group]).sum(-1) + v["D"] * u
        return (y if gate is None else y * gate), h
    train = case["op"] == "scan_train"
    cu = v["cu_host"]
    T, N = cu[-1], len(cu) - 1
    if T * C * S * 8 > 24e9 and train:
        return None
    order = sorted(range(N), key=lambda n: cu[n] - cu[n + 1])  # longest first: the documents alive at step t come first
    length = [cu[n + 1] - cu[n] for n in order]
    start = torch.tensor([cu[n] for n in order], device="cuda")
    h = torch.zeros((N, C, S), dtype=d, device="cuda") if v["h0"] is None else v["h0"][order].clone()
    h0 = h.clone()
    y0 = torch.empty((T, C), dtype=d, device="cuda")
    hs = torch.empty((T, C, S), dtype=d, device="cuda") if train else None
    alive, k = [], N
    for t in range(max(length, default=0)):
        while k and length[k - 1] <= t:
            k -= 1
        alive.append(k)
        r = start[:k] + t
        h[:k] = torch.exp(delta[r][..., None] * A) * h[:k] + (delta[r] * u[r])[..., None] * v["B"][r][:, group]
        y0[r] = (h[:k] * v["Cm"][r][:, group]).sum(-1)
        if train:
            hs[r] = h[:k]
    y0 += v["D"] * u
    back = torch.tensor(sorted(range(N), key=lambda i: order[i]), device="cuda")
    out = dict(y=y0 if gate is None else y0 * gate, ht=h[back])
    if not train:
        return out["y"], out["ht"]
    dy = v["dy"]
    if gate is not None:
        s = torch.sigmoid(v["z"])
        out["dz"] = dy * y0 * (s + v["z"] * s * (1 - s))
        dy = dy * gate
    g = torch.zeros_like(h) if v["dht"] is None else v["dht"][order].clone()
    dB, dC = (torch.zeros((T, G, S), dtype=d, device="cuda") for _ in range(2))
    du, dd = torch.empty_like(u), torch.empty_like(u)
    dA = torch.zeros_like(A)
    for t in range(len(alive) - 1, -1, -1):
        k = alive[t]
        r = start[:k] + t
        g[:k] += dy[r][..., None] * v["Cm"][r][:, group]
        a = torch.exp(delta[r][..., None] * A)
        prev = h0[:k] if t == 0 else hs[r - 1]
        dC[r] = (dy[r][..., None] * hs[r]).view(k, G, C // G, S).sum(2)
        dB[r] = (g[:k] * (delta[r] * u[r])[..., None]).view(k, G, C // G, S).sum(2)
        sB = (g[:k] * v["B"][r][:, group]).sum(-1)
        w = g[:k] * a * prev
        du[r] = delta[r] * sB + v["D"] * dy[r]
        dd[r] = u[r] * sB + (w * A).sum(-1)
        dA += (w * delta[r][..., None]).sum(0)
        g[:k] *= a
    dd *= torch.sigmoid(raw)
    out.update(du=du, ddt=dd, dA=dA, dB=dB, dC=dC, dD=(dy * u).sum(0), ddt_bias=dd.sum(0))
    if v["h0"] is not None:
        out["dh0"] = g[back]
    return out


def work(case):
    op, C = case["op"], case["C"]
    e = _BYTES[case.get("dtype", "bf16")]
    if op.startswith("scan"):
        S, G = case["S"], case["G"]
        lens = [int(n) for n in case["lens"].split(",")] if "lens" in case else [1] * case["N"]
        T, N = sum(lens), len(lens)
        z = int(case["z"])
        data = e * T * C * (3 + z) + 2 * e * T * G * S + 4 * C * (S + 2) + 4 * N * C * S
        flops = 7 * T * C * S
        if op == "scan_step":
            data += 4 * N * C * S
        elif case["h0"]:
            data += 4 * N * C * S
        if op == "scan_train":
            data += e * T * C * (3 + z) + 2 * e * T * G * S + 4 * C * (S + 2) + (8 * N * C * S if case["h0"] else 0)
            flops += 14 * T * C * S
        return {"bytes": data, "flops": flops}
    if op == "conv_step":
        return {"bytes": 2 * case["N"] * C * 8 + 20 * C, "flops": 12 * case["N"] * C}
    if op == "conv_prompt":
        lens = case["lens"].split(",")
        T, N = sum(int(n) for n in lens), len(lens)
        return {"bytes": 4 * T * C + 6 * N * C * (2 if case["halo"] else 1) + 20 * C, "flops": 12 * T * C}
    T, r = case["T"], int(case["res"])
    data, flops = e * T * C * (2 + 2 * r) + 8 * C, 8 * T * C
    if op == "norm_train":
        data, flops = data + e * T * C * (2 + r) + 8 * C, flops + 14 * T * C
    return {"bytes": data, "flops": flops}
