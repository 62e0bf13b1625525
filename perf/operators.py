"""Workloads of the node embedding, the query/key norm with rotation and the
attention among the atoms of a structure: the same inputs through plain torch
operations (``own`` false) or through the library's calls (``own`` true).

Lengths are Angstrom, densities those of condensed matter (about 0.1 atoms
per cubic Angstrom); queries and keys have unit root mean square per head, as
the norm in front of the attention leaves them."""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
DENSITY = 0.1


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # species of the 1000-atom diamond cell -> h0 of a message block
        {"name": "embed-cell", "op": "embed", "back": False, "dtype": "f32", "tokens": 1000, "rows": 95, "channels": 128},
        # gradient of the species table over a training batch: few rows, each very long
        {"name": "embed-species", "op": "embed", "back": True, "dtype": "f32", "tokens": 300000, "rows": 95,
         "channels": 128},
        # a large vocabulary (fragments, tokens), most rows hit seldom or never
        {"name": "embed-vocabulary", "op": "embed", "back": True, "dtype": "bf16", "tokens": 65536, "rows": 50000,
         "channels": 512},
        # one new atom or token: latency
        {"name": "rope-token", "op": "rope", "back": False, "dtype": "bf16", "tokens": 1, "heads_q": 16, "heads_k": 4,
         "head_dim": 64, "n_freq": 32, "interleaved": False},
        # a batch of structures, 128 channels as 4 heads of 32, rotated by position in space
        {"name": "rope-batch", "op": "rope", "back": False, "dtype": "f32", "tokens": 131072, "heads_q": 4, "heads_k": 4,
         "head_dim": 32, "n_freq": 16, "interleaved": True},
        # training step with shared key heads
        {"name": "rope-train", "op": "rope", "back": True, "dtype": "bf16", "tokens": 40001, "heads_q": 16, "heads_k": 4,
         "head_dim": 128, "n_freq": 48, "interleaved": False},
        # the smallest structure: latency
        {"name": "attn-tiny", "op": "attn", "back": False, "dtype": "f32", "segments": 1, "min_q": 32, "max_q": 32,
         "min_k": 0, "max_k": 0, "heads_q": 4, "heads_k": 4, "head_dim": 32, "bias": True, "cap": 0.0, "causal": False},
        # one query per structure over all its atoms (readout, or the next atom to place)
        {"name": "attn-single", "op": "attn", "back": False, "dtype": "bf16", "segments": 16, "min_q": 1, "max_q": 1,
         "min_k": 16, "max_k": 8192, "heads_q": 16, "heads_k": 4, "head_dim": 64, "bias": True, "cap": 0.0,
         "causal": False},
        # a batch of molecules, energy and forces: energy gradient through scores and distances
        {"name": "attn-molecules", "op": "attn", "back": True, "dtype": "f32", "segments": 384, "min_q": 5, "max_q": 120,
         "min_k": 0, "max_k": 0, "heads_q": 8, "heads_k": 8, "head_dim": 16, "bias": True, "cap": 0.0, "causal": False},
        # the 4096-atom cell, forces included
        {"name": "attn-cell", "op": "attn", "back": True, "dtype": "f32", "segments": 1, "min_q": 4096, "max_q": 4096,
         "min_k": 0, "max_k": 0, "heads_q": 4, "heads_k": 4, "head_dim": 32, "bias": True, "cap": 0.0, "causal": False},
        # atoms placed one after another beside a given scaffold (prefix): packed training batch
        {"name": "attn-causal", "op": "attn", "back": True, "dtype": "bf16", "segments": 7, "min_q": 300, "max_q": 2500,
         "min_k": 0, "max_k": 0, "heads_q": 16, "heads_k": 4, "head_dim": 128, "bias": False, "cap": 30.0,
         "causal": True},
        # a large structure in one piece
        {"name": "attn-large", "op": "attn", "back": False, "dtype": "bf16", "segments": 1, "min_q": 16384,
         "max_q": 16384, "min_k": 0, "max_k": 0, "heads_q": 8, "heads_k": 8, "head_dim": 64, "bias": True, "cap": 0.0,
         "causal": False},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "rope", "attn", "attn"])
    dtype, back = rng.choice(["f32", "bf16"]), rng.random() < 0.5
    if op == "embed":
        channels = _log(rng, 5, 1024) if rng.random() < 0.3 else 8 * _log(rng, 1, 128)
        return {"op": op, "back": back, "dtype": dtype, "tokens": _log(rng, 1, min(400000, 40000000 // channels)),
                "rows": _log(rng, 2, 60000), "channels": channels}
    if op == "rope":
        d = rng.choice([16, 24, 32, 48, 64, 80, 96, 128])
        hk = rng.choice([1, 2, 3, 4, 8])
        hq = hk * rng.choice([1, 2, 4])
        n_freq = d // 2 if rng.random() < 0.5 else rng.randint(1, d // 2)
        return {"op": op, "back": back, "dtype": dtype, "tokens": _log(rng, 1, min(140000, 100000000 // ((hq + hk) * d))),
                "heads_q": hq, "heads_k": hk, "head_dim": d, "n_freq": n_freq, "interleaved": rng.random() < 0.5}
    d = rng.choice([16, 24, 32, 48, 64, 96, 128])
    hk = rng.choice([1, 2, 3, 4])
    hq = hk * rng.choice([1, 2, 4])
    causal = rng.random() < 0.4
    bias = rng.random() < 0.5
    cap = rng.choice([0.0, 0.0, 20.0, 50.0])
    kind = rng.choice(["one", "single", "ragged"])
    # pairs * heads * head_dim of the largest listed case is 1.4e11, a third of it for a backward pass in 32 bits
    budget = 1.3e11 if not back else 1.2e10
    longest = int(math.sqrt(budget / (hq * d)))
    if kind == "one":
        n = _log(rng, 1, min(10000, longest))
        seg = {"segments": 1, "min_q": n, "max_q": n, "min_k": 0, "max_k": 0}
    elif kind == "single":
        hi = _log(rng, 64, 16000)
        seg = {"segments": _log(rng, 1, 64), "min_q": 1, "max_q": 1, "min_k": _log(rng, 1, hi), "max_k": hi}
    else:
        hi = _log(rng, 10, min(3000, longest // 2))
        seg = {"segments": max(2, min(_log(rng, 2, 500), int(budget / (hq * d) / hi / hi))),
               "min_q": _log(rng, 1, hi), "max_q": hi, "min_k": 0, "max_k": 0}
        if rng.random() < 0.3 and not causal:
            seg["max_k"] = _log(rng, 1, hi)
            seg["min_k"] = _log(rng, 1, seg["max_k"])
    return {"op": "attn", "back": back, "dtype": dtype, **seg, "heads_q": hq, "heads_k": hk, "head_dim": d, "bias": bias,
            "cap": cap, "causal": causal}


def _lengths(case):
    """Lengths of the segments' queries and keys and of their prefixes, as a
    program that packs a batch has them on the host; the case's own."""
    g = torch.Generator().manual_seed(1000 + 31 * case["segments"] + case["max_q"] + case["max_k"])
    s = case["segments"]
    span = lambda lo, hi: torch.randint(lo, hi + 1, (s,), generator=g).tolist()
    lq = span(case["min_q"], case["max_q"])
    # max_k 0: the keys are the queries' own rows
    lk = span(case["min_k"], case["max_k"]) if case["max_k"] else lq
    prefix = [int(f * n) for f, n in zip(torch.rand(s, generator=g).mul(0.5).tolist(), lk)] if case["causal"] else None
    return lq, lk, prefix


def _pairs(case):
    lq, lk, prefix = _lengths(case)
    if not case["causal"]:
        return sum(a * b for a, b in zip(lq, lk))
    total = 0
    for a, b, p in zip(lq, lk, prefix):
        off = b - a
        # query i sees the first max(prefix, i + off + 1) keys
        i = torch.arange(a)
        total += int(torch.clamp(torch.maximum(i + off + 1, torch.tensor(p)), 0, b).sum())
    return total


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "embed":
        n, c = case["tokens"], case["channels"]
        rows = min(n, case["rows"])
        b, f = rows * c * e + 4 * n + n * c * e, n * c
        if case["back"]:
            b, f = b + n * c * e + 4 * n + case["rows"] * c * 4, 3 * n * c
        return {"bytes": b, "flops": f}
    if case["op"] == "rope":
        el = case["tokens"] * (case["heads_q"] + case["heads_k"]) * case["head_dim"]
        b, f = 2 * el * e + 12 * case["tokens"], 8 * el
        if case["back"]:
            b, f = b + 3 * el * e + 24 * case["tokens"], f + 20 * el
        return {"bytes": b, "flops": f}
    lq, lk, _ = _lengths(case)
    nq, nk, d = sum(lq), sum(lk), case["head_dim"]
    hq, hk = case["heads_q"], case["heads_k"]
    b = 2 * nq * hq * d * e + 2 * nk * hk * d * e + nq * hq * 4 + (12 * (nq + nk) if case["bias"] else 0)
    f = 4 * d * hq * _pairs(case)
    if case["back"]:   # q, out, g and k, v again, their gradients
        b += 4 * nq * hq * d * e + 4 * nk * hk * d * e + nq * hq * 4 + (24 * (nq + nk) if case["bias"] else 0)
        f += 10 * d * hq * _pairs(case)
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------ inputs --

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    normal = lambda *s: torch.randn(s, device=dev, generator=g)
    uniform = lambda *s: torch.rand(s, device=dev, generator=g)
    st = {"case": case}
    if case["op"] == "embed":
        n, r, c = case["tokens"], case["rows"], case["channels"]
        # frequencies fall with the row's rank, as species and tokens do
        st["ids"] = torch.clamp((torch.exp(uniform(n) * math.log(r + 1.0)) - 1.0).to(torch.int32), 0, r - 1)
        st["table"], st["scale"] = normal(r, c).to(dt), math.sqrt(c)
        st["g"] = normal(n, c).to(dt)
    elif case["op"] == "rope":
        n, hq, hk, d = case["tokens"], case["heads_q"], case["heads_k"], case["head_dim"]
        # queries, keys and values come from one projection: rows of (hq + 2 hk) d
        qkv = normal(n, (hq + 2 * hk) * d).to(dt)
        st["q"], st["k"] = qkv[:, :hq * d].view(n, hq, d), qkv[:, hq * d:(hq + hk) * d].view(n, hk, d)
        st["gamma_q"], st["gamma_k"] = 1 + 0.1 * normal(d), 1 + 0.1 * normal(d)
        st["pos"] = uniform(n, 3) * (n / DENSITY) ** (1 / 3)
        # wave vectors in random directions, wavelengths of 2 to 200 Angstrom
        k = normal(case["n_freq"], 3)
        st["freq"] = k / k.norm(dim=1, keepdim=True) * (2 * math.pi / (2 * 100 ** uniform(case["n_freq"], 1)))
        st["g_q"], st["g_k"] = normal(n, hq, d).to(dt), normal(n, hk, d).to(dt)
        st["eps"] = 1e-5
    else:
        lq, lk, prefix = _lengths(case)
        nq, nk = sum(lq), sum(lk)
        hq, hk, d = case["heads_q"], case["heads_k"], case["head_dim"]
        unit = lambda t: t / t.square().mean(-1, keepdim=True).sqrt()
        st["lq"], st["lk"], st["prefix"] = lq, lk, prefix
        st["q"], st["k"] = unit(normal(nq, hq, d)).to(dt), unit(normal(nk, hk, d)).to(dt)
        st["v"], st["g"] = normal(nk, hk, d).to(dt), normal(nq, hq, d).to(dt)
        st["scale"], st["cap"] = 1 / math.sqrt(d), case["cap"]
        st["slope"] = st["pos_q"] = st["pos_k"] = None
        if case["bias"]:
            st["slope"] = 0.5 * 2.0 ** (-6.0 * torch.arange(hq, device=dev, dtype=torch.float32) / hq)
            sides = torch.tensor([(max(a, b) / DENSITY) ** (1 / 3) for a, b in zip(lq, lk)], device=dev)
            box = lambda n, ls: uniform(n, 3) * sides.repeat_interleave(torch.tensor(ls, device=dev))[:, None]
            st["pos_q"] = box(nq, lq)
            st["pos_k"] = box(nk, lk) if case["max_k"] else None   # None: the queries' own
    if own:
        _prepare_own(st)
    return st


def run(state):
    op = state["case"]["op"]
    if own:
        return {"embed": _own_embed, "rope": _own_rope, "attn": _own_attn}[op](state)
    return {"embed": _plain_embed, "rope": _plain_rope, "attn": _plain_attn}[op](state)


# -------------------------------------------------------- the library's calls --

def _prepare_own(st):
    """Descriptors, uploaded segment offsets, outputs and workspaces, as a
    program keeps them between steps."""
    from cartesian_tensor_product_amd import flashcart as fc
    case = st["case"]
    dtype = fc.FC_F32 if case["dtype"] == "f32" else fc.FC_BF16
    new = lambda t: torch.empty(t.shape, dtype=t.dtype, device=t.device)
    f32 = lambda *s: torch.empty(s, device="cuda")
    st["fc"] = fc
    if case["op"] == "embed":
        st["d"] = fc.embed_desc(case["tokens"], case["rows"], case["channels"], st["scale"], dtype)
        st["out"] = new(st["g"])
        if case["back"]:
            st["table_grad"] = f32(case["rows"], case["channels"])
            st["ws"] = fc.workspace(fc.fc_embed_workspace_bytes(st["d"]))
    elif case["op"] == "rope":
        d = st["d"] = fc.qk_rope_desc(case["tokens"], case["heads_q"], case["heads_k"], case["head_dim"], case["n_freq"],
                                      st["eps"], dtype, fc.FC_ROPE_INTERLEAVED if case["interleaved"] else 0)
        st["q_out"], st["k_out"] = new(st["g_q"]), new(st["g_k"])
        if case["back"]:
            st["q_grad"], st["k_grad"] = new(st["g_q"]), new(st["g_k"])
            st["gamma_q_grad"], st["gamma_k_grad"] = new(st["gamma_q"]), new(st["gamma_k"])
            st["pos_grad"] = new(st["pos"])
            st["ws"] = fc.workspace(fc.fc_qk_norm_rope_workspace_bytes(d))
    else:
        offsets = lambda ls: torch.tensor([0] + ls).cumsum(0)
        st["seg"] = fc.Segments(offsets(st["lq"]), offsets(st["lk"]) if case["max_k"] else None, st["prefix"])
        d = st["d"] = fc.attn_desc(sum(st["lq"]), sum(st["lk"]), len(st["lq"]), case["heads_q"], case["heads_k"],
                                   case["head_dim"], st["scale"], st["cap"], dtype,
                                   fc.FC_ATTN_CAUSAL if case["causal"] else 0)
        st["out"], st["lse"] = new(st["q"]), f32(sum(st["lq"]), case["heads_q"])
        st["ws"] = fc.workspace(fc.fc_attention_workspace_bytes(d, 0))
        if case["back"]:
            st["q_grad"], st["k_grad"], st["v_grad"] = new(st["q"]), new(st["k"]), new(st["v"])
            st["slope_grad"] = new(st["slope"]) if case["bias"] else None
            st["pos_q_grad"] = new(st["pos_q"]) if case["bias"] else None
            st["pos_k_grad"] = new(st["pos_k"]) if st["pos_k"] is not None else None
            st["ws_vjp"] = fc.workspace(fc.fc_attention_workspace_bytes(d, 1))


def _own_embed(st):
    fc = st["fc"]
    fc.fc_embed_fwd(st["d"], st["table"], st["ids"], st["out"])
    if not st["case"]["back"]:
        return st["out"]
    fc.fc_embed_vjp(st["d"], st["ids"], st["g"], st["table_grad"], st["ws"])
    return st["out"], st["table_grad"]


def _own_rope(st):
    fc = st["fc"]
    args = (st["d"], st["q"], st["k"], st["gamma_q"], st["gamma_k"], st["pos"], st["freq"])
    fc.fc_qk_norm_rope_fwd(*args, st["q_out"], st["k_out"])
    if not st["case"]["back"]:
        return st["q_out"], st["k_out"]
    fc.fc_qk_norm_rope_vjp(*args, st["g_q"], st["g_k"], st["q_grad"], st["k_grad"], st["gamma_q_grad"],
                           st["gamma_k_grad"], st["pos_grad"], st["ws"])
    return (st["q_out"], st["k_out"], st["q_grad"], st["k_grad"], st["gamma_q_grad"], st["gamma_k_grad"],
            st["pos_grad"])


def _own_attn(st):
    fc = st["fc"]
    args = (st["d"], st["seg"], st["q"], st["k"], st["v"], st["slope"], st["pos_q"], st["pos_k"])
    fc.fc_attention_fwd(*args, st["out"], st["lse"], st["ws"])
    if not st["case"]["back"]:
        return st["out"], st["lse"]
    fc.fc_attention_vjp(*args, st["out"], st["lse"], st["g"], st["q_grad"], st["k_grad"], st["v_grad"],
                        st["slope_grad"], st["pos_q_grad"], st["pos_k_grad"], st["ws_vjp"])
    outs = (st["out"], st["lse"], st["q_grad"], st["k_grad"], st["v_grad"], st["slope_grad"], st["pos_q_grad"],
            st["pos_k_grad"])
    return tuple(t for t in outs if t is not None)


# -------------------------------------------------------------- plain forms --

def _plain_embed(st):
    t = st["table"]
    ids = st["ids"].long()
    out = (t[ids].float() * st["scale"]).to(t.dtype)
    if not st["case"]["back"]:
        return out
    # long sums (every atom of one species): 64 bits; few rows as a product with one-hot columns
    if t.shape[0] <= 256:
        grad = (torch.arange(t.shape[0], device=t.device)[:, None] == ids).double() @ st["g"].double()
    else:
        grad = torch.zeros(t.shape, dtype=torch.float64, device=t.device)
        grad.index_add_(0, ids, st["g"].double())
    return out, (grad * st["scale"]).float()


def _split_pairs(x, r, interleaved):
    """(first, second) of the rotated pairs and what passes unrotated."""
    rot, rest = x[..., :2 * r], x[..., 2 * r:]
    if interleaved:
        return rot[..., 0::2], rot[..., 1::2], rest
    return rot[..., :r], rot[..., r:], rest


def _join_pairs(a, b, rest, interleaved):
    rot = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((rot, rest), -1)


def _plain_rope(st):
    case = st["case"]
    r, il = case["n_freq"], case["interleaved"]
    angle = (st["pos"].double() @ st["freq"].double().T)[:, None, :]   # far positions: 64 bits
    c, s = torch.cos(angle).float(), torch.sin(angle).float()
    outs, grads, gammas, pos_grad = [], [], [], torch.zeros_like(st["pos"])
    for x, gamma, g in ((st["q"], st["gamma_q"], st["g_q"]), (st["k"], st["gamma_k"], st["g_k"])):
        xf = x.float()
        inv = 1.0 / torch.sqrt(xf.square().mean(-1, keepdim=True) + st["eps"])
        y = xf * inv * gamma
        a, b, rest = _split_pairs(y, r, il)
        outs.append(_join_pairs(a * c - b * s, a * s + b * c, rest, il).to(x.dtype))
        if not case["back"]:
            continue
        ga, gb, grest = _split_pairs(g.float(), r, il)
        ya, yb = ga * c + gb * s, gb * c - ga * s
        gy = _join_pairs(ya, yb, grest, il)
        pos_grad += (yb * a - ya * b).sum(1) @ st["freq"]
        gammas.append((gy * xf * inv).sum((0, 1)))
        gg = gy * gamma
        grads.append((inv * gg - xf * inv ** 3 * (gg * xf).mean(-1, keepdim=True)).to(x.dtype))
    return (*outs, *grads, *gammas, pos_grad) if case["back"] else tuple(outs)


def _groups(lq, lk, heads):
    """Runs of consecutive segments whose padded scores stay below 2^29
    elements."""
    out, i = [], 0
    while i < len(lq):
        j, mq, mk = i, 0, 0
        while j < len(lq):
            a, b = max(mq, lq[j]), max(mk, lk[j])
            if j > i and (j + 1 - i) * a * b * heads > 1 << 29:
                break
            mq, mk, j = a, b, j + 1
        out.append((i, j, mq, mk))
        i = j
    return out


def _plain_attn(st):
    case = st["case"]
    hq, hk, d, back = case["heads_q"], case["heads_k"], case["head_dim"], case["back"]
    grp, dev, dt = hq // hk, st["q"].device, st["q"].dtype
    lq, lk = st["lq"], st["lk"]
    oq, ok = [0], [0]
    for a, b in zip(lq, lk):
        oq.append(oq[-1] + a)
        ok.append(ok[-1] + b)
    q, k, v = st["q"].float(), st["k"].float(), st["v"].float()
    pq = st["pos_q"]
    pk = pq if st["pos_k"] is None else st["pos_k"]
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device=dev)
    if back:
        g = st["g"].float()
        gq, gk, gv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        if case["bias"]:
            gs, gpq, gpk = torch.zeros_like(st["slope"]), torch.zeros_like(pq), torch.zeros_like(pk)
    for s0, s1, mq, mk in _groups(lq, lk, 1):
        ns = s1 - s0
        # padded row indices and which of them are real
        tq, tk = torch.tensor(lq[s0:s1], device=dev), torch.tensor(lk[s0:s1], device=dev)
        iq, ik = torch.arange(mq, device=dev), torch.arange(mk, device=dev)
        vq, vk = iq < tq[:, None], ik < tk[:, None]
        rq = torch.where(vq, iq + torch.tensor(oq[s0:s1], device=dev)[:, None], 0)
        rk = torch.where(vk, ik + torch.tensor(ok[s0:s1], device=dev)[:, None], 0)
        keep = vq[:, :, None] & vk[:, None, :]
        if case["causal"]:
            pre = torch.tensor(st["prefix"][s0:s1], device=dev)[:, None, None]
            keep &= (ik <= iq[:, None] + (tk - tq)[:, None, None]) | (ik < pre)
        if case["bias"]:
            diff = pq[rq][:, :, None, :] - pk[rk][:, None, :, :]
            dist = diff.square().sum(-1).sqrt()
            pull = torch.zeros_like(dist)
        step = max(1, (1 << 29) // max(1, ns * mq * mk))   # heads at a time
        for h0 in range(0, hq, step):
            hs = list(range(h0, min(hq, h0 + step)))
            hks = [h // grp for h in hs]
            qs = q[:, hs][rq].transpose(1, 2)
            ks = k[:, hks][rk].transpose(1, 2)
            vs = v[:, hks][rk].transpose(1, 2)
            sc = (qs @ ks.transpose(-1, -2)) * st["scale"]
            if case["cap"]:
                th = torch.tanh(sc / st["cap"])
                sc = th * st["cap"]
            if case["bias"]:
                sl = st["slope"][hs][:, None, None]
                sc = sc - sl * dist[:, None]
            sc = torch.where(keep[:, None], sc, -math.inf)
            top = sc.amax(-1, keepdim=True).clamp_min(-3e38)
            p = torch.exp(sc - top)
            total = p.sum(-1, keepdim=True)
            p = p / total.clamp_min(1e-38)
            hidx = torch.tensor(hs, device=dev)
            where_q = rq[vq]
            out[where_q[:, None], hidx] = (p @ vs).transpose(1, 2)[vq]
            lse[where_q[:, None], hidx] = (top + torch.log(total)).squeeze(-1).transpose(1, 2)[vq]
            if not back:
                continue
            go = torch.where(vq[:, None, :, None], g[:, hs][rq].transpose(1, 2), 0)
            dp = go @ vs.transpose(-1, -2)
            ds = p * (dp - (p * dp).sum(-1, keepdim=True))
            if case["bias"]:
                gs[hs] -= (ds * dist[:, None]).sum((0, 2, 3))
                pull -= (sl * ds).sum(1)
            if case["cap"]:
                ds = ds * (1 - th * th)
            gq[where_q[:, None], hidx] = ((ds @ ks) * st["scale"]).transpose(1, 2)[vq]
            where_k = rk[vk]
            dk, dv = (ds.transpose(-1, -2) @ qs) * st["scale"], p.transpose(-1, -2) @ go
            for n, hkv in enumerate(hks):   # shared key heads add up
                gk[where_k, hkv] += dk[:, n][vk]
                gv[where_k, hkv] += dv[:, n][vk]
        if back and case["bias"]:
            w = torch.where(dist > 0, pull / dist, 0)[..., None] * diff
            gpq[rq[vq]] += w.sum(2)[vq]
            gpk[rk[vk]] -= w.sum(1)[vk]
    if not back:
        return out.to(dt), lse
    outs = [out.to(dt), lse, gq.to(dt), gk.to(dt), gv.to(dt)]
    if case["bias"]:
        outs += [gs, gpq + gpk] if st["pos_k"] is None else [gs, gpq, gpk]
    return tuple(outs)


# ------------------------------------------------- definitions in 64 bits --

def exact(case, seed):
    global own
    kept, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    return {"embed": _exact_embed, "rope": _exact_rope, "attn": _exact_attn}[case["op"]](case, st)


def _exact_embed(case, st):
    # the lookup as products with one-hot rows, some tokens at a time; the
    # gradient as differences of the running sum over the sorted tokens
    t, ids = st["table"].double(), st["ids"]
    rows = torch.arange(case["rows"], device=t.device, dtype=torch.int32)
    step = max(1, (1 << 27) // case["rows"])
    out = torch.cat([st["scale"] * ((i[:, None] == rows).double() @ t) for i in ids.split(step)])
    if not case["back"]:
        return out
    order = torch.argsort(ids)
    run = torch.cat((torch.zeros_like(t[:1]), st["g"][order].double().cumsum(0)))
    ends = torch.searchsorted(ids[order].contiguous(), rows, right=True)
    starts = torch.searchsorted(ids[order].contiguous(), rows)
    return out, st["scale"] * (run[ends] - run[starts])


def _exact_rope(case, st):
    r, il, d = case["n_freq"], case["interleaved"], case["head_dim"]
    leaf = lambda t: t.detach().double().requires_grad_(case["back"])
    q, k, wq, wk, pos = (leaf(st[n]) for n in ("q", "k", "gamma_q", "gamma_k", "pos"))
    freq = st["freq"].double()
    # the pair's member indices, and a rotation as a product of complex numbers
    first = torch.arange(r, device=q.device) * (2 if il else 1)
    second = first + (1 if il else r)
    turn = torch.exp(1j * (pos[:, None, :] * freq).sum(-1))[:, None, :]

    def one(x, w):
        y = w * x * torch.rsqrt((x * x).sum(-1, keepdim=True) / d + st["eps"])
        z = torch.complex(y[..., first], y[..., second]) * turn
        return y.index_copy(-1, first, z.real).index_copy(-1, second, z.imag)

    oq, ok = one(q, wq), one(k, wk)
    if not case["back"]:
        return oq, ok
    loss = (oq * st["g_q"].double()).sum() + (ok * st["g_k"].double()).sum()
    grads = torch.autograd.grad(loss, (q, k, wq, wk, pos))
    return (oq.detach(), ok.detach(), *grads)


def _exact_attn(case, st):
    if _pairs(case) * case["heads_q"] > 3e9 or case["segments"] * case["heads_q"] > 12000:
        return None
    back, bias = case["back"], case["bias"]
    leaf = lambda t: None if t is None else t.detach().double().requires_grad_(back)
    names = ["q", "k", "v"] + (["slope", "pos_q"] if bias else []) + (["pos_k"] if st["pos_k"] is not None else [])
    x = {n: leaf(st[n]) for n in names}
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    lse = torch.zeros(out.shape[:2], dtype=torch.float64, device=out.device)
    sums = {n: torch.zeros_like(t) for n, t in x.items()}
    grp = case["heads_q"] // case["heads_k"]
    a = b = 0
    for s, (nq, nk) in enumerate(zip(st["lq"], st["lk"])):
        own_keys = st["pos_k"] is None
        # as many heads at once as fit, one shared key head at least per step
        heads = max(1, min(case["heads_q"], int(2 ** 27 / max(1, nq * nk))))
        for h0 in range(0, case["heads_q"], heads):
            h = torch.arange(h0, min(case["heads_q"], h0 + heads), device=out.device)
            part = {"q": x["q"][a:a + nq], "k": x["k"][b:b + nk], "v": x["v"][b:b + nk]}
            if bias:
                part["slope"], part["pos_q"] = x["slope"], x["pos_q"][a:a + nq]
                if not own_keys:
                    part["pos_k"] = x["pos_k"][b:b + nk]
            part = {n: t.detach().requires_grad_(back) for n, t in part.items()}
            qh, kh, vh = (part["q"][:, h].permute(1, 0, 2), part["k"][:, h // grp].permute(1, 2, 0).contiguous(),
                          part["v"][:, h // grp].permute(1, 0, 2).contiguous())
            u = torch.bmm(qh, kh) * st["scale"]
            if st["cap"]:
                u = st["cap"] * torch.tanh(u / st["cap"])
            if bias:
                pk = part["pos_q"] if own_keys else part["pos_k"]
                sq = sum((part["pos_q"][:, None, i] - pk[None, :, i]) ** 2 for i in range(3))
                near = sq == 0
                u = u - part["slope"][h, None, None] * torch.where(near, 0.0, torch.where(near, 1.0, sq).sqrt())
            if case["causal"]:
                seen = torch.ones(nq, nk, dtype=torch.bool, device=u.device).tril(nk - nq)
                seen[:, :st["prefix"][s]] = True
                u = u.masked_fill(~seen, -math.inf)
            z = torch.logsumexp(u, -1)
            o = torch.bmm(torch.exp(u - z[..., None]), vh)
            out[a:a + nq, h] = o.detach().permute(1, 0, 2)
            lse[a:a + nq, h] = z.detach().t()
            if back:
                gr = torch.autograd.grad((o * st["g"][a:a + nq, h].permute(1, 0, 2).double()).sum(), list(part.values()))
                for n, t in zip(part, gr):
                    at = (a, nq) if n in ("q", "pos_q") else (b, nk)
                    if n == "slope":
                        sums[n] += t
                    else:
                        sums[n][at[0]:at[0] + at[1]] += t
        a, b = a + nq, b + nk
    return (out, lse, *(sums[n] for n in names)) if back else (out, lse)
