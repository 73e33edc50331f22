"""The attention block of a decode step for many continuations of one prompt: rotary positions with the cache append,
attention of a batch that shares a prefix, and grouped matrix-vector products with 4-bit weights.

``own = False`` computes the operators in elementary torch operations; ``own = True`` calls the framework's kernels on the
same inputs.  Head shapes, widths and vocabulary sizes are those of the repository's workloads, or generic odd ones.
"""
import math

import torch

if torch.cuda.is_available():
    torch.backends.cuda.matmul.allow_tf32 = False

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    rope = dict(op="rope", layout="half", theta=10000.0, scaling="none", factor=1.0, pad=False)
    q4 = dict(op="q4")
    attn = dict(op="attn")
    return [
        # one token of one sequence: the call's latency (1.5B-class heads)
        dict(rope, name="rope_one_token", T=1, seqs=1, hq=16, hkv=16, hd=128, rot=128, cap=1024, dtype="f32", cache="bf16",
             maxpos=700),
        # a decode step of 193 continuations, some slots of the batch unused, interleaved pairs on 3/4 of the head
        dict(rope, name="rope_batch_193", T=193, seqs=193, hq=32, hkv=8, hd=128, rot=96, cap=256, dtype="f32", cache="bf16",
             maxpos=32768, layout="interleaved", pad=True),
        # an 8K-token prompt written at far positions of a context stretched 8 times (YaRN)
        dict(rope, name="rope_prompt_8k", T=8192, seqs=1, hq=32, hkv=8, hd=128, rot=128, cap=8192, dtype="bf16", cache="bf16",
             maxpos=262144, scaling="yarn", factor=8.0),
        # the 9B-class model's Q, K and V projections of one token, norm fused
        dict(q4, name="q4_qkv_1", rows="4096,1024,1024", cols=4096, M=1, dtype="f32", group=128, scales="bf16", zeros=False,
             norm=True),
        # the 4B-class model's vocabulary head for one token
        dict(q4, name="q4_head_1", rows="151936", cols=2560, M=1, dtype="f32", group=128, scales="bf16", zeros=False, norm=True),
        # gate and up of the 9B-class model for eight continuations, finer groups with zero points
        dict(q4, name="q4_gate_up_8", rows="12288,12288", cols=4096, M=8, dtype="bf16", group=64, scales="bf16", zeros=True,
             norm=False),
        # odd rows, smallest groups, fp32 scales, five fp32 vectors (the 1.5B-class down projection's width)
        dict(q4, name="q4_ragged_5", rows="2049,37", cols=5632, M=5, dtype="f32", group=32, scales="f32", zeros=True, norm=False),
        # one short question, one sequence: latency
        dict(attn, name="attn_short_1", B=1, P=37, cap=16, hq=16, hkv=16, hd=128, dtype="f32"),
        # odd batch, odd prefix, every head its own keys, fp32 queries
        dict(attn, name="attn_mha_17", B=17, P=1111, cap=300, hq=16, hkv=16, hd=128, dtype="f32"),
        # 32 continuations of the 9B-class workload's 2048-token prompt
        dict(attn, name="attn_b32_p2048", B=32, P=2048, cap=512, hq=32, hkv=8, hd=128, dtype="bf16"),
        # 64 continuations of the 4B-class workload's 32K-token prompt
        dict(attn, name="attn_b64_p32k", B=64, P=32768, cap=256, hq=32, hkv=8, hd=128, dtype="bf16"),
        # a wide batch over a long system prompt: the products bound it
        dict(attn, name="attn_b256_p8k", B=256, P=8192, cap=512, hq=32, hkv=8, hd=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_HEADS = [(16, 16, 128), (32, 8, 128), (28, 4, 128), (14, 2, 64), (5, 5, 64), (8, 1, 128)]


def draw(rng):
    op = rng.choice(["rope", "q4", "q4", "attn", "attn"])
    hq, hkv, hd = rng.choice(_HEADS)
    if op == "rope":
        T = _log(rng, 1, 8192)
        seqs = min(T, _log(rng, 1, 256))
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        per = -(-T // seqs)
        return dict(op=op, T=T, seqs=seqs, hq=hq, hkv=hkv, hd=hd, rot=rng.choice([hd, hd // 2, hd // 4, hd - 6]),
                    cap=per + rng.randrange(0, 200), dtype=rng.choice(["f32", "bf16"]), cache=rng.choice(["bf16", "bf16", "f32"]),
                    layout=rng.choice(["half", "interleaved"]), theta=rng.choice([10000.0, 500000.0]), scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]), maxpos=_log(rng, 9000, 1000000),
                    pad=T > 3 and rng.random() < 0.4)
    if op == "q4":
        group = rng.choice([32, 64, 128])
        cols = group * max(1, _log(rng, 256, 12288) // group)
        rows, left = [], 151936 * 2560 // cols
        for _ in range(rng.choice([1, 1, 2, 3])):
            rows.append(_log(rng, 1, max(1, min(32000, left // 3))))
        return dict(op=op, rows=",".join(map(str, rows)), cols=cols, M=_log(rng, 1, 32), dtype=rng.choice(["f32", "bf16"]),
                    group=group, scales=rng.choice(["bf16", "f32"]), zeros=rng.random() < 0.5, norm=rng.random() < 0.5)
    B = _log(rng, 1, 256)
    P = _log(rng, 1, min(32768, 64 * 32768 // B))
    cap = _log(rng, 1, min(2048, 131072 // B))
    return dict(op=op, B=B, P=P, cap=cap, hq=hq, hkv=hkv, hd=hd, dtype=rng.choice(["f32", "bf16"]))


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _ints(g, lo, hi, n):
    return torch.randint(lo, hi, (n,), generator=g, device="cuda")


def _frequencies(c):
    """Angle per position of each pair, and the factor on cos and sin (64-bit)."""
    r, base, s = c["rot"], float(c["theta"]), float(c["factor"])
    i = torch.arange(r // 2, dtype=torch.float64)
    if c["scaling"] == "ntk" and r > 2:
        base = base * s ** (r / (r - 2))
    f = base ** (-2.0 * i / r)
    if c["scaling"] == "linear":
        return f / s, 1.0
    if c["scaling"] == "yarn":
        at = lambda beta: r * math.log(YARN_CONTEXT / (2 * math.pi * beta)) / (2 * math.log(base))  # noqa: E731
        lo = min(max(math.floor(at(32.0)), 0), r // 2 - 1)
        hi = min(max(math.ceil(at(1.0)), 0), r // 2 - 1)
        keep = 1 - ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f / s * (1 - keep) + f * keep, 0.1 * math.log(s) + 1.0
    return f, 1.0


YARN_CONTEXT = 32768  # the context that the stretched model was made for


def _prepare_rope(c, g):
    T, S, hq, hkv, hd, cap = c["T"], c["seqs"], c["hq"], c["hkv"], c["hd"], c["cap"]
    per = -(-T // S)
    qkv = _rn(g, T, (hq + 2 * hkv) * hd, dtype=DT[c["dtype"]])  # one row a token, as the fused projection leaves it
    q, k, v = qkv.split([hq * hd, hkv * hd, hkv * hd], dim=1)
    i = torch.arange(T, device="cuda")
    seq, step = i % S, i // S
    start = _ints(g, 0, max(1, c["maxpos"] - per), S)
    base = _ints(g, 0, cap - per + 1, S)
    pos, slot = (start[seq] + step).int(), (base[seq] + step).int()
    if c["pad"]:  # unused places of the batch: rotated, not appended
        slot = torch.where((i % 7 == 3), torch.full_like(slot, -1), slot)
    st = dict(c=c, q=q.view(T, hq, hd), k=k.view(T, hkv, hd), v=v.view(T, hkv, hd), pos=pos, seq=seq.int(), slot=slot,
              q_out=torch.empty(T, hq, hd, dtype=DT[c["dtype"]], device="cuda"),
              kc=_rn(g, S, hkv, cap, hd, dtype=DT[c["cache"]]), vc=_rn(g, S, hkv, cap, hd, dtype=DT[c["cache"]]))
    if own:  # the plan that a program makes once
        import speculative_pipeline_decoding_gb300 as spd
        st["rope"] = spd.Rope(hd, rot_dim=c["rot"], layout=c["layout"], theta=c["theta"], scaling=c["scaling"],
                              factor=c["factor"], original_context=YARN_CONTEXT)
    else:
        f, m = _frequencies(c)
        st["freq"], st["mscale"] = f.cuda(), m
    return st


def _quantise(w, group, sdt, zeros):
    """Round-to-nearest 4-bit codes of w with one scale (and zero point) for `group` columns."""
    rows, cols = w.shape
    wg = w.view(rows, cols // group, group)
    if zeros:
        hi, lo = wg.amax(2).clamp(min=0), wg.amin(2).clamp(max=0)
        s = ((hi - lo) / 15).to(sdt)
        sf = s.float().clamp(min=1e-20)
        z = torch.round(-lo / sf).clamp(0, 15)
    else:
        s = (wg.abs().amax(2) / 7).to(sdt)
        sf = s.float().clamp(min=1e-20)
        z = torch.full_like(sf, 8)
    code = (torch.round(wg / sf[..., None]) + z[..., None]).clamp(0, 15).to(torch.uint8).view(rows, cols)
    return code[:, 0::2] | (code[:, 1::2] << 4), s, z.to(torch.uint8) if zeros else None


def _prepare_q4(c, g):
    st = dict(c=c, W=[])
    for rows in map(int, c["rows"].split(",")):
        W = torch.randn(rows, c["cols"], generator=g, device="cuda").mul_(0.02)
        st["W"].append(_quantise(W, c["group"], DT[c["scales"]], c["zeros"]))
        del W
    x = torch.randn(c["M"], c["cols"], generator=g, device="cuda")
    x[:, _ints(g, 0, c["cols"], max(1, c["cols"] // 500))] *= 20  # the few large channels of a residual stream
    st["x"] = x.to(DT[c["dtype"]])
    st["nw"] = 1 + 0.1 * torch.randn(c["cols"], generator=g, device="cuda") if c["norm"] else None
    st["y"] = [torch.empty(c["M"], int(r), dtype=DT[c["dtype"]], device="cuda") for r in c["rows"].split(",")]
    if own:  # the weights as a program keeps them, laid out once
        import speculative_pipeline_decoding_gb300 as spd
        st["packed"] = [spd.q4_pack(*w) for w in st["W"]]
    return st


def _prepare_attn(c, g):
    B, P, cap, hq, hkv, hd = (c[k] for k in ("B", "P", "cap", "hq", "hkv", "hd"))
    bf = torch.bfloat16
    # queries of a little more than unit size, so that some keys weigh more than others, as after q and k norms
    st = dict(c=c, q=(1.5 * _rn(g, B, hq, hd)).to(DT[c["dtype"]]), pk=_rn(g, hkv, P, hd, dtype=bf), pv=_rn(g, hkv, P, hd, dtype=bf),
              kc=_rn(g, B, hkv, cap, hd, dtype=bf), vc=_rn(g, B, hkv, cap, hd, dtype=bf), lens=_ints(g, 0, cap + 1, B).int())
    st["out"] = torch.empty_like(st["q"])
    st["lse"] = torch.empty(B, hq, device="cuda")
    if own:  # the workspace that a program keeps
        import speculative_pipeline_decoding_gb300 as spd
        n = spd.shared_prefix_attention_workspace_bytes(B, hq, hkv, hd, P)
        st["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    return st


def prepare(case, seed):
    g = _gen(seed)
    return {"rope": _prepare_rope, "q4": _prepare_q4, "attn": _prepare_attn}[case["op"]](case, g)


# ---------------------------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------------------------
def _rotate(x, cos, sin, rot, layout):
    """x [T, heads, hd] in 32 bits, cos and sin [T, 1, rot / 2]."""
    y = x.clone()
    if layout == "half":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y[..., : rot // 2], y[..., rot // 2: rot] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    return y


def _run_rope(st):
    c = st["c"]
    if own:
        import speculative_pipeline_decoding_gb300 as spd
        spd.rope_append(st["rope"], st["q"], st["q_out"], st["pos"], k=st["k"], v=st["v"], k_cache=st["kc"], v_cache=st["vc"],
                        slot=st["slot"], seq=st["seq"])
        return {"q": st["q_out"], "k_cache": st["kc"], "v_cache": st["vc"]}
    angle = st["pos"].double()[:, None, None] * st["freq"]
    cos, sin = (angle.cos() * st["mscale"]).float(), (angle.sin() * st["mscale"]).float()
    q = _rotate(st["q"].float(), cos, sin, c["rot"], c["layout"]).to(st["q"].dtype)
    k = _rotate(st["k"].float(), cos, sin, c["rot"], c["layout"]).to(st["kc"].dtype)
    v = st["v"].to(st["vc"].dtype)
    # tokens without a slot repeat the write of the first token that has one
    valid = st["slot"] >= 0
    src = torch.where(valid, torch.arange(c["T"], device="cuda"), valid.int().argmax())
    seq, slot = st["seq"].long()[src], st["slot"].long()[src]
    st["kc"][seq, :, slot] = k[src]
    st["vc"][seq, :, slot] = v[src]
    return {"q": q, "k_cache": st["kc"], "v_cache": st["vc"]}


def _dequant(W, group):
    codes, s, z = W
    code = torch.stack([codes & 15, codes >> 4], dim=2).view(codes.shape[0], -1, group)
    return ((code.float() - (z.float()[..., None] if z is not None else 8.0)) * s.float()[..., None]).view(codes.shape[0], -1)


def _run_q4(st):
    c = st["c"]
    if own:
        import speculative_pipeline_decoding_gb300 as spd
        spd.q4_gemv(st["packed"], [st["x"]] * len(st["y"]), st["y"], norm_weight=st["nw"], eps=1e-6)
        return st["y"]
    x = st["x"].float()
    if st["nw"] is not None:
        x = x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6) * st["nw"]
    return [(x @ _dequant(W, c["group"]).T).to(st["x"].dtype) for W in st["W"]]


def _run_attn(st):
    c = st["c"]
    B, P, hq, hkv, hd = (c[k] for k in ("B", "P", "hq", "hkv", "hd"))
    if own:
        import speculative_pipeline_decoding_gb300 as spd
        spd.shared_prefix_attention(st["q"], st["pk"], st["pv"], P, st["kc"], st["vc"], st["lens"], st["out"], st["ws"],
                                    lse=st["lse"])
        return {"out": st["out"], "lse": st["lse"]}
    G = hq // hkv
    q = st["q"].float().view(B, hkv, G, hd) / math.sqrt(hd)
    s1 = (q.transpose(0, 1).reshape(hkv, B * G, hd) @ st["pk"].float().transpose(1, 2)).view(hkv, B, G, P).transpose(0, 1)
    s2 = q @ st["kc"].float().transpose(2, 3)
    there = torch.arange(c["cap"], device="cuda") < st["lens"][:, None]
    s2 = torch.where(there[:, None, None], s2, float("-inf"))
    m = torch.maximum(s1.amax(3), s2.amax(3))[..., None]
    p1, p2 = (s1 - m).exp(), (s2 - m).exp()
    total = p1.sum(3) + p2.sum(3)
    o = (p1.transpose(0, 1).reshape(hkv, B * G, P) @ st["pv"].float()).view(hkv, B, G, hd).transpose(0, 1)
    o = (o + p2 @ st["vc"].float()) / total[..., None]
    return {"out": o.reshape(B, hq, hd).to(st["q"].dtype), "lse": (m[..., 0] + total.log()).reshape(B, hq)}


def run(state):
    return {"rope": _run_rope, "q4": _run_q4, "attn": _run_attn}[state["c"]["op"]](state)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------
def work(case):
    c = case
    size = {"f32": 4, "bf16": 2}
    if c["op"] == "rope":
        e, ce = size[c["dtype"]], size[c["cache"]]
        kept = c["T"] - (len(range(3, c["T"], 7)) if c["pad"] else 0)  # the others' keys and values are not read
        return {"bytes": c["T"] * (2 * c["hq"] * c["hd"] * e + 12) + kept * 2 * c["hkv"] * c["hd"] * (e + ce),
                "flops": 3 * c["rot"] * (c["T"] * c["hq"] + kept * c["hkv"])}
    if c["op"] == "q4":
        rows, e = sum(map(int, c["rows"].split(","))), size[c["dtype"]]
        groups = rows * c["cols"] // c["group"]
        return {"bytes": rows * c["cols"] // 2 + groups * (size[c["scales"]] + (1 if c["zeros"] else 0)) + c["M"] * (c["cols"] + rows) * e
                + (c["cols"] * 4 if c["norm"] else 0), "flops": 2 * rows * c["cols"] * c["M"]}
    keys = c["B"] * (c["cap"] // 2)  # lengths are uniform in 0..cap
    return {"bytes": (c["P"] + keys) * 2 * c["hkv"] * c["hd"] * 2 + c["B"] * c["hq"] * (2 * c["hd"] * size[c["dtype"]] + 4) + 4 * c["B"],
            "flops": 4 * (c["B"] * c["P"] + keys) * c["hq"] * c["hd"]}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------
def _exact_rope(c, st):
    rot, half = c["rot"], c["rot"] // 2
    f, m = _frequencies(c)
    turn = torch.polar(torch.full((c["T"], half), float(m), dtype=torch.float64, device="cuda"),
                       st["pos"].double()[:, None] * f.cuda())

    def rotated(x):
        x = x.double().clone()
        head = x[..., :rot]
        pairs = head.unflatten(-1, (2, half)).transpose(-1, -2) if c["layout"] == "half" else head.unflatten(-1, (half, 2))
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None])
        x[..., :rot] = (z.transpose(-1, -2) if c["layout"] == "half" else z).flatten(-2)
        return x

    kc, vc = st["kc"].double(), st["vc"].double()
    at = (st["slot"] >= 0).nonzero()[:, 0]
    where = (st["seq"].long()[at], slice(None), st["slot"].long()[at])
    kc[where], vc[where] = rotated(st["k"])[at], st["v"].double()[at]
    return {"q": rotated(st["q"]), "k_cache": kc, "v_cache": vc}


def _exact_q4(c, st):
    x = st["x"].double()
    if st["nw"] is not None:
        x = st["nw"].double() * x / ((x * x).sum(1, keepdim=True) / c["cols"] + 1e-6).sqrt()
    out = []
    for codes, s, z in st["W"]:
        y = torch.empty(c["M"], codes.shape[0], dtype=torch.float64, device="cuda")
        for r in range(0, codes.shape[0], 16384):
            part = codes[r: r + 16384]
            w = torch.empty(part.shape[0], c["cols"], dtype=torch.float64, device="cuda")
            w[:, 0::2], w[:, 1::2] = (part % 16).double(), (part // 16).double()
            w -= z[r: r + 16384].double().repeat_interleave(c["group"], 1) if z is not None else 8
            w *= s[r: r + 16384].double().repeat_interleave(c["group"], 1)
            y[:, r: r + 16384] = torch.einsum("mc,rc->mr", x, w)
        out.append(y)
    return out


def _exact_attn(c, st):
    B, hq, hkv = c["B"], c["hq"], c["hkv"]
    out = torch.empty(B, hq, c["hd"], dtype=torch.float64, device="cuda")
    lse = torch.empty(B, hq, dtype=torch.float64, device="cuda")
    lens = st["lens"].tolist()
    for h in range(hkv):
        pk, pv = st["pk"][h].double(), st["pv"][h].double()
        heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
        for b in range(B):
            k = torch.cat([pk, st["kc"][b, h, : lens[b]].double()])
            v = torch.cat([pv, st["vc"][b, h, : lens[b]].double()])
            s = st["q"][b, heads].double() @ k.T / c["hd"] ** 0.5
            lse[b, heads] = s.logsumexp(1)
            out[b, heads] = torch.softmax(s, 1) @ v
    return {"out": out, "lse": lse}


def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "q4": _exact_q4, "attn": _exact_attn}[case["op"]](case, st)
