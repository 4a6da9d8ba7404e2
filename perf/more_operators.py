"""Cases and plain forms of the operators that serve trees of drafted tokens from a paged cache.

Four operators, in the order of a generation step:

plan    block tables and slot maps from the requests' lengths: every sequence is given the
        pages its new tokens need, from a ring of free ones, and returns those it no longer
        needs; every new row learns its slot in the pool and its rotary position (in a tree
        of drafted tokens the position goes by a token's depth).
append  new keys (normalised, rotated at the given positions) and values written to the given
        slots of the pools.
tree    attention of a tree of drafted tokens over the paged cache: each sees every cached
        position, its ancestors and itself.
keep    the accepted path of the tree, its keys and values moved to the positions right behind
        the cached ones.

`run` with own = False computes the plain form: elementary torch operations in fp32 (fp64 for
angles), rounded once.
"""
import math
import random

import torch

own = False

BASE = 10000.0
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token for each of 64 running requests; every 16th needs a page
        dict(name="plan_step", op="plan", B=64, lo=100, hi=8000, new_lo=1, new_hi=1, page=16, tree=False, surplus=0, short=False, pad=0),
        # a step of drafted trees: pages that the rejected tokens held before go back, and the pool runs short
        dict(name="plan_trees_short", op="plan", B=48, lo=0, hi=3000, new_lo=5, new_hi=24, page=16, tree=True, surplus=3, short=True, pad=29),
        # prompts of mixed length enter
        dict(name="plan_prompts", op="plan", B=200, lo=0, hi=0, new_lo=33, new_hi=4096, page=64, tree=False, surplus=1, short=False, pad=100),
        # 16 trees of 16 drafted tokens into the cache of the 12/4-head model
        dict(name="append_trees", op="append", N=256, Hkv=4, D=64, page=16, norm=True, half=False, top=8192, fused=False),
        # a batch of prompts, their rows inside a fused projection's, some refused a place
        dict(name="append_prompts", op="append", N=16381, Hkv=4, D=64, page=64, norm=True, half=True, top=4096, fused=True),
        # the smallest call: one sequence, eight drafted tokens, a short context (latency)
        dict(name="tree_one", op="tree", B=1, Tq=8, lo=129, hi=129, Hq=12, Hkv=4, D=64, page=16, norm=False, ragged=False, idle=0, fp32=False),
        # the small model's heads, odd short contexts, trees of different sizes, idle slots
        dict(name="tree_odd", op="tree", B=33, Tq=13, lo=1, hi=1111, Hq=4, Hkv=2, D=32, page=16, norm=True, ragged=True, idle=2, fp32=False),
        # a serving batch: trees of 16 tokens on contexts around 8192
        dict(name="tree_batch", op="tree", B=16, Tq=16, lo=4100, hi=12288, Hq=12, Hkv=4, D=64, page=64, norm=True, ragged=False, idle=0, fp32=False),
        # a larger batch with 32 tokens each, contexts up to 4096
        dict(name="tree_wide", op="tree", B=64, Tq=32, lo=700, hi=4096, Hq=16, Hkv=4, D=64, page=32, norm=True, ragged=True, idle=1, fp32=False),
        # the largest tree on one very long context
        dict(name="tree_long", op="tree", B=1, Tq=64, lo=131001, hi=131001, Hq=16, Hkv=4, D=64, page=128, norm=False, ragged=False, idle=0, fp32=True),
        # one sequence's accepted path in one layer (latency)
        dict(name="keep_one", op="keep", B=1, Tq=8, hi=500, Hkv=4, D=64, page=16),
        # 64 trees of 32 tokens, the 16 layers of the 12/4-head model in one pool
        dict(name="keep_layers", op="keep", B=64, Tq=32, hi=300, Hkv=64, D=64, page=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "tree", "tree", "tree", "keep"])
    page = rng.choice([16, 32, 64, 128, 256])
    D = rng.choice([64, 64, 32])
    if op == "plan":
        B = _log(rng, 1, 500)
        tree = rng.random() < 0.5
        hi = 64 if tree else _log(rng, 1, max(1, 400000 // B))
        return dict(op=op, B=B, lo=0, hi=_log(rng, 1, 20000), new_lo=rng.randint(0, hi), new_hi=hi, page=page, tree=tree,
                    surplus=rng.choice([0, 2, 5]), short=rng.random() < 0.3, pad=rng.choice([0, 7]))
    Hq, Hkv = rng.choice([(12, 4), (16, 4), (4, 2), (4, 4), (8, 1), (6, 3)])
    if op == "append":
        return dict(op=op, N=_log(rng, 1, 16000), Hkv=Hkv, D=D, page=page, norm=rng.random() < 0.5, half=rng.random() < 0.5,
                    top=_log(rng, 64, 100000), fused=rng.random() < 0.5)
    if op == "keep":
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, Tq=rng.randint(1, 32), hi=rng.randint(1, 300), Hkv=Hkv * rng.choice([1, 8]), D=D, page=page)
    B = _log(rng, 1, 100)
    hi = _log(rng, 1, max(16, 100000 // B))
    return dict(op=op, B=B, Tq=rng.randint(1, 64 if B < 16 else 32), lo=rng.randint(0, hi), hi=hi, Hq=Hq, Hkv=Hkv, D=D, page=page,
                norm=rng.random() < 0.5, ragged=rng.random() < 0.5, idle=rng.choice([0, 0, 1]) if B > 1 else 0,
                fp32=rng.random() < 0.3)


def _spread(B, lo, hi):
    """B whole numbers spread over lo .. hi, the same for every seed."""
    if B == 1:
        return [hi]
    return [lo + ((hi - lo) * ((i * 61803 + 7) % 100003)) // 100002 for i in range(B)]


def _nodes(c):
    """Tokens of every sequence's tree."""
    if c.get("ragged") and c["B"] > 1:
        return _spread(c["B"], 1, c["Tq"])
    return [c["Tq"]] * c["B"]


def _contexts(c):
    """Cached positions of every sequence before its tree; None: an idle slot of the batch."""
    n = _spread(c["B"], c["lo"], c["hi"])
    for i in range(c["idle"]):
        n[(i * 7 + 1) % c["B"]] = None
    return n


def _accepted(c):
    """(accepted tokens, how many of them are in place already) of every sequence."""
    m = [max(1, x) for x in _spread(c["B"], 0, c["Tq"] // 2)]
    return [(x, max(min(x, i % 3), 2 * x - c["Tq"])) for i, x in enumerate(m)]


# ------------------------------------------------------------------ inputs
def _parents(r, n):
    """A tree of n tokens: the first hangs on the context, each of the others on one a little earlier."""
    return [-1 if t == 0 else r.randint(max(-1 if r.random() < 0.1 else 0, t - 6), t - 1) for t in range(n)]


def _pages(P, seed):
    return torch.randperm(P, generator=torch.Generator().manual_seed(int(seed)), dtype=torch.int32)


def _table(need, width, order):
    table = torch.full((len(need), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    r = random.Random(int(seed))

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    def weight(D):
        return (1 + 0.1 * torch.randn(D, generator=g, device=dev)).to(torch.bfloat16)

    s = dict(case=c)
    page = c["page"]
    if c["op"] == "plan":
        B = c["B"]
        kv, new = _spread(B, c["lo"], c["hi"]), _spread(B, c["new_lo"], c["new_hi"])
        want = [-(-(k + n) // page) for k, n in zip(kv, new)]
        # pages held: those of the cached positions, and for some what a longer past left them
        held = [-(-k // page) + (c["surplus"] if i % 3 == 1 else 0) for i, k in enumerate(kv)]
        need = sum(max(0, w - h) for w, h in zip(want, held))
        free = max(1, need * 2 // 3 if c["short"] else need + 17)
        P = sum(held) + free
        order = _pages(P, seed)
        s["table"] = _table(held, max(1, max(want + held)), order).to(dev)
        first = P - free // 2 - 1  # the free pages go round the end of the ring
        ring = torch.zeros(P, dtype=torch.int32)
        ring[(first + torch.arange(free)) % P] = order[sum(held):]
        s["ring"], s["span"] = ring.to(dev), ints([first, free])
        s["held"], s["kv"], s["new"] = ints(held), ints(kv), ints(new)
        s["rows"] = max(1, sum(new) + c["pad"])
        s["parents"] = ints([_parents(r, c["new_hi"]) for _ in range(B)]) if c["tree"] else None
        return s
    D, Hkv = c["D"], c["Hkv"]
    if c["op"] == "append":
        N = c["N"]
        kv = normal(N, 2 * Hkv, D)
        s["k"], s["v"] = kv[:, :Hkv], kv[:, Hkv:]
        if not c["fused"]:
            s["k"], s["v"] = s["k"].contiguous(), s["v"].contiguous()
        s["kw"] = weight(D) if c["norm"] else None
        # a sequence's rows lie side by side, its pages anywhere; a few rows were refused a place
        P = N // page + 9
        row = torch.arange(N)
        slots = _pages(P, seed)[row // page + 4] * page + (row % page).to(torch.int32)
        slots[row % 97 == 5] = -1
        s["slots"] = slots.to(dev)
        s["pos"] = ints([r.randrange(c["top"]) for _ in range(N)])
    else:
        B = c["B"]
        if c["op"] == "tree":
            ctx, nodes = _contexts(c), _nodes(c)
            total = [0 if x is None else x + n for x, n in zip(ctx, nodes)]
            s["q"] = normal(B, c["Tq"], c["Hq"], D)
            s["qw"] = weight(D) if c["norm"] else None
            s["parents"] = ints([_parents(r, c["Tq"]) for _ in range(B)])
        else:
            nodes = [c["Tq"]] * B
            total = [x + c["Tq"] for x in _spread(B, 0, c["hi"])]
            path = []
            for m, there in _accepted(c):
                # the first tokens of the path are in place, the others lie behind the places they
                # move to (a tree level by level, its levels wider than the path is long)
                rest = sorted(r.sample(range(m, c["Tq"]), m - there))
                path.append(list(range(there)) + rest + [-1] * (c["Tq"] - m))
            s["path"], s["m"] = ints(path), ints([m for m, _ in _accepted(c)])
        s["nodes"], s["len"] = ints(nodes), ints(total)
        need = [-(-n // page) for n in total]
        P = sum(need) + 3
        s["table"] = _table(need, max(1, max(need)), _pages(P, seed)).to(dev)
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


def _reach(parents):
    """[B, T, T] truth values: token t's ancestors and itself."""
    T = parents.shape[-1]
    x = (torch.arange(T, device=parents.device) == parents[..., None]) | torch.eye(T, dtype=torch.bool, device=parents.device)
    x = x.float()
    for _ in range(max(1, (T - 1).bit_length())):
        x = ((x @ x) > 0).float()
    return x > 0


def _plain_plan(s):
    page, table, ring = s["case"]["page"], s["table"], s["ring"]
    kv, new, held = s["kv"].long(), s["new"].long(), s["held"].long()
    first, count = s["span"].long()
    P = ring.numel()
    want = (kv + new + page - 1) // page
    need, give = (want - held).clamp(min=0), (held - want).clamp(min=0)
    run = need.cumsum(0)
    ok = (need == 0) | (run <= count)
    got = torch.where(ok, need, 0)
    i = torch.arange(table.shape[1], device=table.device)
    j = i - held[:, None]
    mine = (j >= 0) & (j < got[:, None])
    page_of = ring[(first + (run - need)[:, None] + j) % P]
    back = (i >= want[:, None]) & (i < held[:, None])
    to = (first + count + (give.cumsum(0) - give)[:, None] + i - want[:, None]) % P
    ring[to[back]] = table[back]
    table.copy_(torch.where(mine, page_of, table))
    taken, returned = got.sum(), give.sum()
    span = torch.stack(((first + taken) % P, count - taken + returned)).int()
    cu = torch.cat((new.new_zeros(1), new.cumsum(0)))
    row = torch.arange(s["rows"], device=table.device)
    b = torch.searchsorted(cu[1:], row, right=True).clamp(max=len(kv) - 1)
    t = row - cu[b]
    at = kv[b] + t
    real = row < cu[-1]
    where = (at // page).clamp(max=table.shape[1] - 1)
    slot = torch.where(real & ok[b], table[b, where].long() * page + at % page, -1)
    if s["parents"] is not None:
        depth = _reach(s["parents"]).sum(-1) - 1
        at = kv[b] + depth[b, t.clamp(max=depth.shape[1] - 1)]
    pos = torch.where(real, at, 0)
    total = kv + torch.where(ok, new, 0)
    return table, ring, torch.where(ok, want, held).int(), span, total.int(), cu.int(), slot.int(), pos.int()


def _plain_append(s):
    c = s["case"]
    on = s["slots"] >= 0
    slot = s["slots"][on].long()
    k = _rotate(_norm(s["k"][on], s["kw"]), s["pos"][on], c["half"], c["D"])
    s["kp"][slot // c["page"], :, slot % c["page"]] = k.to(torch.float16)
    s["vp"][slot // c["page"], :, slot % c["page"]] = s["v"][on]
    return s["kp"], s["vp"]


def _plain_tree(s):
    c = s["case"]
    B, Tq, Hq, Hkv, D = c["B"], c["Tq"], c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    n, nodes = s["len"].long(), s["nodes"].long()
    ctx = n - nodes
    reach = _reach(s["parents"])
    pos = ctx[:, None] + reach.sum(-1) - 1
    q = _rotate(_norm(s["q"], s["qw"]), pos.clamp(min=0), False, D)
    q = q.view(B, Tq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Tq, D)
    t = s["table"].long().clamp(min=0)
    k = s["kp"][t].permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D).float()
    x = (q @ k.transpose(-1, -2)) / math.sqrt(D)
    del k
    L = x.shape[-1]
    j = torch.arange(L, device=n.device) - ctx[:, None]  # the place in the tree of every position
    see = torch.gather(reach, 2, j.clamp(0, Tq - 1)[:, None].expand(B, Tq, L))
    see = (j < 0)[:, None] | (see & (j < nodes[:, None])[:, None])
    see &= ((torch.arange(Tq, device=n.device) < nodes[:, None]) & (ctx >= 0)[:, None])[..., None]
    x = x.masked_fill(~see.repeat(1, G, 1)[:, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m.clamp(min=-1e30))
    del x, see
    z = p.sum(-1, keepdim=True)
    v = s["vp"][t].permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D).float()
    o = (p @ v) / torch.where(z > 0, z, 1.0)
    lse = (m + z.log()).squeeze(-1)
    o = o.view(B, Hkv, G, Tq, D).permute(0, 3, 1, 2, 4).reshape(B, Tq, Hq, D)
    return o.to(torch.float32 if c["fp32"] else torch.bfloat16), lse.view(B, Hq, Tq)


def _plain_keep(s):
    c = s["case"]
    page = c["page"]
    ctx = s["len"].long() - c["Tq"]
    i = torch.arange(c["Tq"], device=ctx.device)
    b, i = torch.nonzero(i < s["m"][:, None], as_tuple=True)
    src, dst = ctx[b] + s["path"][b, i], ctx[b] + i
    for pool in (s["kp"], s["vp"]):
        rows = pool[s["table"][b, src // page].long(), :, src % page]
        pool[s["table"][b, dst // page].long(), :, dst % page] = rows
    return s["kp"], s["vp"], (ctx + s["m"]).int()


def run(s):
    if own:
        return _own(s)
    return {"plan": _plain_plan, "append": _plain_append, "tree": _plain_tree, "keep": _plain_keep}[s["case"]["op"]](s)


def _own(s):
    from causal_gqa_attention_flashattention_gb300 import binding as nb
    c = s["case"]
    if c["op"] == "plan":
        p = nb.paged_plan(s["table"], s["ring"], s["held"], s["span"], s["kv"], s["new"], s["rows"], c["page"], parents=s["parents"])
        return s["table"], s["ring"], p.held, p.span, p.kv_len, p.cu_new, p.slots, p.positions
    if c["op"] == "append":
        nb.kv_append_slots(s["k"], s["v"], s["kp"], s["vp"], s["slots"], s["pos"], c["top"], k_weight=s["kw"], eps=EPS,
                           rope_base=BASE, rope_half=c["half"])
        return s["kp"], s["vp"]
    if c["op"] == "tree":
        return nb.attn_decode_tree(s["q"], s["kp"], s["vp"], s["table"], s["len"], s["parents"], tree_len=s["nodes"],
                                   q_weight=s["qw"], eps=EPS, rope_base=BASE,
                                   o_dtype=torch.float32 if c["fp32"] else torch.bfloat16)
    n = nb.kv_keep_paged(s["kp"], s["vp"], s["table"], s["len"], s["nodes"], s["path"], s["m"])
    return s["kp"], s["vp"], n


# ------------------------------------------------------------------ the least work of a pass
def work(c):
    page = c["page"]
    if c["op"] == "plan":
        kv, new = _spread(c["B"], c["lo"], c["hi"]), _spread(c["B"], c["new_lo"], c["new_hi"])
        n = sum(new)
        pages = sum(new) // page  # about: each is read in the ring and written to a table
        trees = 4 * c["B"] * c["new_hi"] if c["tree"] else 0
        # lengths, pages held (in and out), row starts; a slot and a position for every row
        return {"bytes": 24 * len(kv) + 8 * pages + 8 * (n + c["pad"]) + trees, "flops": 4 * n}
    D, Hkv = c["D"], c["Hkv"]
    if c["op"] == "append":
        n = c["N"] - len(range(5, c["N"], 97))
        return {"bytes": 8 * n * Hkv * D + 8 * c["N"], "flops": (8 if c["norm"] else 3) * n * Hkv * D}
    if c["op"] == "keep":
        moved = sum(m - there for m, there in _accepted(c))
        return {"bytes": 8 * moved * Hkv * D + 12 * c["B"] + 4 * sum(m for m, _ in _accepted(c)), "flops": moved}
    seen = [(x, n) for x, n in zip(_contexts(c), _nodes(c)) if x is not None]
    keys, table = sum(x + n for x, n in seen), sum(-(-(x + n) // page) for x, n in seen)
    rows = c["B"] * c["Tq"] * c["Hq"]
    out = (4 if c["fp32"] else 2) * D * rows + 4 * rows
    # every token: its context, and of its tree at least itself
    pairs = sum((x + 1) * n for x, n in seen)
    return {"bytes": 4 * D * Hkv * keys + 2 * D * rows + out + 4 * table + 4 * c["B"] * (c["Tq"] + 2),
            "flops": 4 * D * c["Hq"] * pairs}


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
    if c["op"] == "plan":
        return None  # whole numbers
    s = prepare(c, seed)
    D, Hkv, page = c["D"], c["Hkv"], c["page"]
    dev = s["kp"].device
    if c["op"] == "append":
        kp, vp = s["kp"].double(), s["vp"].double()
        k = _turn64(_unit64(s["k"], s["kw"]), s["pos"][:, None], c["half"])
        slots = s["slots"].long()
        for h in range(Hkv):
            flat = slots.clamp(min=0)
            at = (flat // page, torch.full_like(flat, h), flat % page)
            for pool, rows in ((kp, k[:, h]), (vp, s["v"][:, h].double())):
                pool[tuple(x[slots >= 0] for x in at)] = rows[slots >= 0]
        return kp, vp
    if c["op"] == "keep":
        kp, vp = s["kp"].double(), s["vp"].double()
        table, path, lens = s["table"].tolist(), s["path"].tolist(), []
        for b, (n, m) in enumerate(zip(s["len"].tolist(), s["m"].tolist())):
            first = n - c["Tq"]
            lens.append(first + m)
            for i in range(m):
                src, dst = first + path[b][i], first + i
                for pool in (kp, vp):
                    pool[table[b][dst // page], :, dst % page] = pool[table[b][src // page], :, src % page]
        return kp, vp, None
    B, Tq, Hq = c["B"], c["Tq"], c["Hq"]
    G = Hq // Hkv
    o = torch.zeros((B, Tq, Hq, D), dtype=torch.float64, device=dev)
    lse = torch.full((B, Hq, Tq), -math.inf, dtype=torch.float64, device=dev)
    parents = s["parents"].tolist()
    for b, (n, nodes) in enumerate(zip(s["len"].tolist(), s["nodes"].tolist())):
        if n == 0:
            continue
        pages = s["table"][b, :-(-n // page)].long()
        k = s["kp"][pages].transpose(0, 1).reshape(Hkv, -1, D)[:, :n].double()
        v = s["vp"][pages].transpose(0, 1).reshape(Hkv, -1, D)[:, :n].double()
        first = n - nodes
        see = torch.zeros((nodes, n), dtype=torch.bool)
        see[:, :first] = True
        depth = []
        for t in range(nodes):
            depth.append(-1)
            at = t
            while at >= 0:
                see[t, first + at] = True
                depth[t] += 1
                at = parents[b][at]
        pos = first + torch.tensor(depth, device=dev)
        q = _turn64(_unit64(s["q"][b, :nodes], s["qw"]), pos[:, None], False).view(nodes, Hkv, G, D)
        see = see.to(dev)
        for h in range(Hkv):
            x = torch.einsum("tgd,nd->tgn", q[:, h], k[h]) / math.sqrt(D)
            x = x.masked_fill(~see[:, None], -math.inf)
            lse[b, h * G:(h + 1) * G, :nodes] = torch.logsumexp(x, -1).T
            o[b, :nodes, h * G:(h + 1) * G] = torch.einsum("tgn,nd->tgd", torch.softmax(x, -1), v[h])
    return o, lse
