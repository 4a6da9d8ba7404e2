"""Cases and plain forms of the operators around the paged key/value cache.

Four operators, in the order a model uses them:

norm_rope       RMS norm of every query and key head, then the rotary embedding, in
                one pass; the rotated fp16 q and k start the attention's workspace.
norm_rope_grad  its backward: from the attention's gradients of the normalised q and k
                to those of q, k and the two norm weights.
append          new keys (normalised, rotated) and values written into the pages of a
                paged cache, for a ragged batch of new tokens.
decode, prefix  attention of the newest tokens of every sequence over the paged cache,
                each sequence with its own length; `prefix` is the same call for a batch
                whose sequences share their first pages, which are read once for all.

`run` with own = False computes the plain form: elementary torch operations in
fp32 (fp64 for angles and for sums over every row of a batch), rounded once.
"""
import math

import torch

own = False

BASE = 10000.0
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one training step's queries and keys of the 12/4-head model: all of a batch of 16 x 512
        dict(name="norm_rope_train", op="norm_rope", B=16, T=512, Hq=12, Hkv=4, D=64, half=False, fused=False),
        # the small 4/2-head model on an odd length, q and k still inside the fused projection's rows
        dict(name="norm_rope_small_fused", op="norm_rope", B=2, T=77, Hq=4, Hkv=2, D=32, half=True, fused=True),
        # the same training step's way back, bf16 gradients
        dict(name="norm_rope_grad_train", op="norm_rope_grad", B=16, T=512, Hq=12, Hkv=4, D=64, fp32=False, fused=False),
        # fp32 gradients of the 16/4-head shape, odd length
        dict(name="norm_rope_grad_odd", op="norm_rope_grad", B=5, T=1021, Hq=16, Hkv=4, D=64, fp32=True, fused=True),
        # a generation step: one new token for each of 64 sequences with up to 8192 cached positions
        dict(name="append_step", op="append", B=64, lo=1, hi=1, past=8191, Hkv=4, D=64, page=16, norm=True, half=False, pad=0),
        # prompts of mixed length going into the cache, padded to a multiple of rows
        dict(name="append_prompts", op="append", B=23, lo=3, hi=1500, past=0, Hkv=4, D=64, page=64, norm=True, half=True, pad=37),
        # the smallest call: one sequence, one new token, a short context (latency)
        dict(name="decode_one", op="decode", B=1, Tq=1, lo=129, hi=129, Hq=12, Hkv=4, D=64, page=16, norm=False, prefix=0, idle=0),
        # a serving batch of ragged contexts around 8192
        dict(name="decode_batch", op="decode", B=16, Tq=1, lo=4100, hi=12288, Hq=12, Hkv=4, D=64, page=64, norm=True, prefix=0, idle=0),
        # one very long context
        dict(name="decode_long", op="decode", B=1, Tq=1, lo=131001, hi=131001, Hq=16, Hkv=4, D=64, page=128, norm=False, prefix=0, idle=0),
        # five drafted tokens a sequence, short odd contexts, idle slots, the small model's heads
        dict(name="decode_draft_odd", op="decode", B=33, Tq=5, lo=3, hi=1111, Hq=4, Hkv=2, D=32, page=16, norm=True, prefix=0, idle=2),
        # 64 chats on one system prompt
        dict(name="prefix_chat", op="prefix", B=64, Tq=1, lo=1, hi=512, Hq=12, Hkv=4, D=64, page=64, norm=True, prefix=8192, idle=1),
        # a large batch on one long document
        dict(name="prefix_document", op="prefix", B=128, Tq=1, lo=5, hi=1024, Hq=16, Hkv=4, D=64, page=16, norm=False, prefix=16384, idle=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_grad", "append", "decode", "decode", "prefix"])
    Hq, Hkv = rng.choice([(12, 4), (16, 4), (4, 2), (4, 4), (8, 1), (6, 3)])
    D = rng.choice([64, 64, 32])
    page = rng.choice([16, 32, 64, 128, 256])
    if op in ("norm_rope", "norm_rope_grad"):
        rows = _log(rng, 8, 8192)
        B = min(rows, rng.choice([1, 2, 3, 7, 16]))
        c = dict(op=op, B=B, T=max(1, rows // B), Hq=Hq, Hkv=Hkv, D=D, fused=rng.random() < 0.5)
        if op == "norm_rope":
            c["half"] = rng.random() < 0.5
        else:
            c["fp32"] = rng.random() < 0.5
        return c
    if op == "append":
        B = _log(rng, 1, 200)
        hi = _log(rng, 1, max(1, 16384 // B))
        return dict(op=op, B=B, lo=rng.randint(0 if B > 1 else 1, hi), hi=hi, past=_log(rng, 1, 4096), Hkv=Hkv, D=D, page=page,
                    norm=rng.random() < 0.5, half=rng.random() < 0.5, pad=rng.choice([0, 0, 5]))
    if op == "decode":
        B = _log(rng, 1, 128)
        hi = _log(rng, 1, max(16, 100000 // B))
        G = Hq // Hkv
        Tq = rng.choice([1, 1, 1, 2, 3, 4, 7])
        return dict(op=op, B=B, Tq=min(Tq, 32 // G, hi), lo=rng.randint(1, hi), hi=hi, Hq=Hq, Hkv=Hkv, D=D, page=page,
                    norm=rng.random() < 0.5, prefix=0, idle=rng.choice([0, 0, 1]) if B > 1 else 0)
    B = _log(rng, 2, 128)
    prefix = max(1, _log(rng, 64, 16384) // page) * page
    hi = _log(rng, 1, 1000)
    return dict(op=op, B=B, Tq=min(hi, rng.choice([1, 1, 1, 2, 3])), lo=rng.randint(1, hi), hi=hi, Hq=Hq, Hkv=Hkv, D=D, page=page,
                norm=rng.random() < 0.5, prefix=prefix, idle=rng.choice([0, 0, 1]))


def _spread(B, lo, hi):
    """B whole numbers spread over lo .. hi, the same for every seed."""
    if B == 1:
        return [hi]
    return [lo + ((hi - lo) * ((i * 61803 + 7) % 100003)) // 100002 for i in range(B)]


def _lengths(c):
    """Positions of every sequence with its newest tokens; idle slots of the batch have none."""
    n = [c["prefix"] + max(x, c["Tq"]) for x in _spread(c["B"], c["lo"], c["hi"])]
    for i in range(c["idle"]):
        n[(i * 7 + 1) % c["B"]] = 0
    return n


# ------------------------------------------------------------------ inputs
def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    def weight(D):
        return (1 + 0.1 * torch.randn(D, generator=g, device=dev)).to(torch.bfloat16)

    s = dict(case=c)
    D, Hkv = c["D"], c["Hkv"]
    if c["op"] in ("norm_rope", "norm_rope_grad"):
        B, T, Hq = c["B"], c["T"], c["Hq"]
        # activations of a few different sizes, as a projection gives them
        size = torch.exp(0.5 * torch.randn((B, T, Hq + 2 * Hkv, 1), generator=g, device=dev))
        qkv = (torch.randn((B, T, Hq + 2 * Hkv, D), generator=g, device=dev) * size).to(torch.bfloat16)
        s["q"], s["k"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv]
        if not c["fused"]:
            s["q"], s["k"] = s["q"].contiguous(), s["k"].contiguous()
        s["qw"], s["kw"] = weight(D), weight(D)
        if c["op"] == "norm_rope_grad":
            t = torch.float32 if c["fp32"] else torch.bfloat16
            s["gq"], s["gk"] = normal(B, T, Hq, D, dtype=t), normal(B, T, Hkv, D, dtype=t)
        return s
    page, B = c["page"], c["B"]
    if c["op"] == "append":
        new = _spread(B, c["lo"], c["hi"])
        past = [(c["past"] * (i + 1)) // B for i in range(B)]
        total = [a + b for a, b in zip(past, new)]
        shared = 0
        N = sum(new) + c["pad"]
        s["k"], s["v"] = normal(N, Hkv, D), normal(N, Hkv, D)
        cu = [0]
        for x in new:
            cu.append(cu[-1] + x)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        s["pos0"] = torch.tensor(past, dtype=torch.int32, device=dev)
        s["rows"] = cu[-1]
        s["kw"] = weight(D) if c["norm"] else None
    else:
        total = _lengths(c)
        shared = c["prefix"] // page
        s["q"] = normal(B, c["Tq"], c["Hq"], D)
        s["qw"] = weight(D) if c["norm"] else None
        s["len"] = torch.tensor(total, dtype=torch.int32, device=dev)
    need = [-(-n // page) for n in total]
    mine = [max(0, n - shared) for n in need]
    P = shared + sum(mine) + 3
    order = torch.randperm(P, generator=torch.Generator().manual_seed(int(seed)), dtype=torch.int32)
    width = max(1, max(need), shared)
    table = torch.zeros((B, width), dtype=torch.int32)
    at = shared
    for b in range(B):
        table[b, :shared] = order[:shared]
        table[b, shared:shared + mine[b]] = order[at:at + mine[b]]
        at += mine[b]
    s["table"] = table.to(dev)
    s["shared"] = order[:shared].to(dev) if shared else None
    s["kp"] = normal(P, Hkv, page, D, dtype=torch.float16)  # the rotated keys
    s["vp"] = normal(P, Hkv, page, D)
    return s


# ------------------------------------------------------------------ plain forms
def _rotate(x, pos, half, D):
    """Rotary embedding of x [..., H, D] at positions pos [...]; the pairs leave side by side."""
    inv = BASE ** (-torch.arange(0, D, 2, device=x.device, dtype=torch.float64) / D)
    ang = pos.to(torch.float64).unsqueeze(-1) * inv
    c, n = ang.cos().float().unsqueeze(-2), ang.sin().float().unsqueeze(-2)
    a, b = (x[..., :D // 2], x[..., D // 2:]) if half else (x[..., 0::2], x[..., 1::2])
    return torch.stack((a * c - b * n, a * n + b * c), -1).flatten(-2)


def _norm(x, w):
    x = x.float()
    if w is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _plain_norm_rope(s):
    c = s["case"]
    pos = torch.arange(c["T"], device=s["q"].device).expand(c["B"], c["T"])
    return tuple(_rotate(_norm(x, w), pos, c["half"], c["D"]).to(torch.float16)
                 for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])))


def _plain_grad_one(x, w, g):
    xf, gf = x.float(), g.float()
    r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + EPS)
    n = xf * r
    wg = gf * w.float()
    dx = r * (wg - n * (wg * n).mean(-1, keepdim=True))
    return dx.to(g.dtype), (gf * n).sum((0, 1, 2), dtype=torch.float64).float()


def _plain_append(s):
    c, n = s["case"], s["rows"]
    row = torch.arange(n, device=s["k"].device)
    seq = torch.searchsorted(s["cu"][1:].contiguous(), row.to(torch.int32), right=True)
    pos = s["pos0"][seq].long() + row - s["cu"][seq].long()
    page = s["table"][seq, pos // c["page"]].long()
    slot = pos % c["page"]
    k = _rotate(_norm(s["k"][:n], s["kw"]), pos, c["half"], c["D"])
    s["kp"][page, :, slot] = k.to(torch.float16)
    s["vp"][page, :, slot] = s["v"][:n]
    return s["kp"], s["vp"]


def _plain_decode(s):
    c = s["case"]
    B, Tq, Hq, Hkv, D = c["B"], c["Tq"], c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    n = s["len"].long()
    pos = n[:, None] - Tq + torch.arange(Tq, device=n.device)
    q = _rotate(_norm(s["q"], s["qw"]), pos.clamp(min=0), False, D)
    q = q.view(B, Tq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Tq, D)
    t = s["table"].long()
    k = s["kp"][t].permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D).float()
    x = (q @ k.transpose(-1, -2)) / math.sqrt(D)
    del k
    see = torch.arange(x.shape[-1], device=n.device) <= pos.repeat(1, G)[:, None, :, None]
    x = x.masked_fill(~see, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m.clamp(min=-1e30))
    del x, see
    z = p.sum(-1, keepdim=True)
    v = s["vp"][t].permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D).float()
    o = (p @ v) / torch.where(z > 0, z, 1.0)
    lse = (m + z.log()).squeeze(-1)
    o = o.view(B, Hkv, G, Tq, D).permute(0, 3, 1, 2, 4).reshape(B, Tq, Hq, D)
    return o.to(torch.bfloat16), lse.view(B, Hq, Tq)


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        return _own(s)
    if op == "norm_rope":
        return _plain_norm_rope(s)
    if op == "norm_rope_grad":
        dq, dqw = _plain_grad_one(s["q"], s["qw"], s["gq"])
        dk, dkw = _plain_grad_one(s["k"], s["kw"], s["gk"])
        return dq, dk, dqw, dkw
    if op == "append":
        return _plain_append(s)
    return _plain_decode(s)


def _own(s):
    from causal_gqa_attention_flashattention_gb300 import binding as nb
    c = s["case"]
    op = c["op"]
    if op == "norm_rope":
        ws = nb.qk_norm(s["q"], s["k"], s["qw"], s["kw"], eps=EPS, rope_base=BASE, rope_half=c["half"])
        return nb.rotated_qk(ws, c["B"], c["T"], c["Hq"], c["Hkv"], c["D"])
    if op == "norm_rope_grad":
        return nb.qk_norm_bwd(s["q"], s["k"], s["qw"], s["kw"], s["gq"], s["gk"], eps=EPS)
    if op == "append":
        nb.kv_append_paged(s["k"], s["v"], s["kp"], s["vp"], s["table"], s["pos0"], cu_new=s["cu"], k_weight=s["kw"],
                           eps=EPS, rope_base=BASE, rope_half=c["half"])
        return s["kp"], s["vp"]
    return nb.attn_decode_paged(s["q"], s["kp"], s["vp"], s["table"], s["len"], q_weight=s["qw"], eps=EPS, rope_base=BASE,
                                prefix_table=s["shared"], prefix_len=c["prefix"])


# ------------------------------------------------------------------ the least work of a pass
def work(c):
    D, Hkv = c["D"], c["Hkv"]
    if c["op"] in ("norm_rope", "norm_rope_grad"):
        n = c["B"] * c["T"] * (c["Hq"] + Hkv) * D
        if c["op"] == "norm_rope":
            return {"bytes": 4 * n + 4 * D, "flops": 10 * n}  # read bf16, write fp16
        e = 4 if c["fp32"] else 2
        return {"bytes": (2 + 2 * e) * n + 12 * D, "flops": 12 * n}  # read x and the gradient, write the gradient
    if c["op"] == "append":
        n = sum(_spread(c["B"], c["lo"], c["hi"])) * Hkv * D
        return {"bytes": 8 * n + 8 * c["B"] + 4, "flops": (8 if c["norm"] else 3) * n}
    G, Tq, page = c["Hq"] // Hkv, c["Tq"], c["page"]
    seen = _lengths(c)
    keys = c["prefix"] + sum(max(0, n - c["prefix"]) for n in seen)  # the shared positions are read once
    table = sum(-(-n // page) for n in seen)
    rows = c["B"] * Tq * c["Hq"]
    return {"bytes": 4 * D * Hkv * keys + 4 * D * rows + 4 * rows + 4 * table + 4 * c["B"],
            "flops": 4 * D * G * Tq * Hkv * sum(seen)}


# ------------------------------------------------------------------ the definition in 64 bits
def _turn64(x, pos, half):
    """x [..., D] as complex pairs times exp(i pos theta), in 64 bits."""
    D = x.shape[-1]
    z = torch.complex(x[..., :D // 2], x[..., D // 2:]) if half else torch.view_as_complex(x.reshape(*x.shape[:-1], D // 2, 2).contiguous())
    theta = torch.exp(torch.arange(D // 2, device=x.device, dtype=torch.float64) * (-2.0 / D * math.log(BASE)))
    ang = pos.double()[..., None] * theta
    return torch.view_as_real(z * torch.polar(torch.ones_like(ang), ang)).reshape(x.shape)


def _unit64(x, w):
    x = x.double()
    return x if w is None else x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()


def exact(c, seed):
    s = prepare(c, seed)
    D = c["D"]
    if c["op"] == "norm_rope":
        pos = torch.arange(c["T"], device=s["q"].device).view(1, -1, 1)
        return tuple(_turn64(_unit64(x, w), pos, c["half"]) for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])))
    if c["op"] == "norm_rope_grad":
        out, dws = [], []
        for x, w, g in ((s["q"], s["qw"], s["gq"]), (s["k"], s["kw"], s["gk"])):
            x, w, g = x.double(), w.double(), g.double()
            q = x.pow(2).sum(-1, keepdim=True) / D + EPS
            # y_i = w_i x_i q^(-1/2);  dq/dx_j = 2 x_j / D
            out.append(g * w / q.sqrt() - x / (D * q * q.sqrt()) * (g * w * x).sum(-1, keepdim=True))
            dws.append((g * x / q.sqrt()).reshape(-1, D).sum(0))
        return out[0], out[1], dws[0], dws[1]
    if c["op"] == "append":
        kp, vp = s["kp"].double(), s["vp"].double()
        cu, first = s["cu"].tolist(), s["pos0"].tolist()
        for b in range(c["B"]):
            if cu[b] == cu[b + 1]:
                continue
            pos = torch.arange(first[b], first[b] + cu[b + 1] - cu[b], device=kp.device)
            k = _turn64(_unit64(s["k"][cu[b]:cu[b + 1]], s["kw"]), pos[:, None], c["half"])
            where = s["table"][b].long()[pos // c["page"]]
            kp[where, :, pos % c["page"]] = k
            vp[where, :, pos % c["page"]] = s["v"][cu[b]:cu[b + 1]].double()
        return kp, vp
    B, Tq, Hq, Hkv = c["B"], c["Tq"], c["Hq"], c["Hkv"]
    G = Hq // Hkv
    o = torch.zeros((B, Tq, Hq, D), dtype=torch.float64, device=s["q"].device)
    lse = torch.full((B, Hq, Tq), -math.inf, dtype=torch.float64, device=o.device)
    for b, n in enumerate(s["len"].tolist()):
        if n == 0:
            continue
        pages = s["table"][b, :-(-n // c["page"])].long()
        k = s["kp"][pages].transpose(0, 1).reshape(Hkv, -1, D)[:, :n].double()
        v = s["vp"][pages].transpose(0, 1).reshape(Hkv, -1, D)[:, :n].double()
        for t in range(Tq):
            at = n - Tq + t
            if at < 0:
                continue
            q = _turn64(_unit64(s["q"][b, t], s["qw"]), torch.full((1,), at, device=o.device), False).view(Hkv, G, D)
            x = torch.einsum("hgd,hnd->hgn", q, k[:, :at + 1]) / math.sqrt(D)
            lse[b, :, t] = torch.logsumexp(x, -1).reshape(Hq)
            o[b, t] = torch.einsum("hgn,hnd->hgd", torch.softmax(x, -1), v[:, :at + 1]).reshape(Hq, D)
    return o, lse
