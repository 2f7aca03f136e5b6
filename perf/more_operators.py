"""The operators of a step with drafted tokens over the paged cache, as they are measured.

A step of generation writes n rows for every sequence behind what its cache
holds.  They are the nodes of a tree of drafted tokens: ``parents`` names each
row's parent among its sequence's rows (-1: none), row 0 is the root, the last
token that is certain.  A sequence of ``lens`` positions holds its nodes in the
last n of them, in row order.

* rotary   rotary positions of q and k: a node's position is the number of
           cached positions plus its depth in the tree;
* tree     softmax attention of the nodes over the cached positions and over
           their own ancestors (themselves included);
* verify   which branch of the tree the target's probabilities accept, given
           random numbers, and the token that follows it;
* keep     the accepted nodes' keys and values move to the first of the new
           positions, in several layers' caches at once.

``run`` computes them in elementary torch operations, or, where ``own`` is
true, calls the framework's operators.
"""
import math

import torch

own = False


def listed():
    return [
        # one step of 64 sequences, a chain of two rows each: latency alone
        _rotary("rotary_step", "bf16", 64, 2, 0.0, 4000, 0.8, False, 0, 32, 8, 128, 128, 0, "interleaved", False, 1, False),
        # prompts of four sequences, frequencies scaled for long contexts
        _rotary("rotary_prompts", "bf16", 4, 4096, 0.4, 60000, 0.5, False, 3, 32, 8, 128, 128, 0, "half", True, 1, False),
        # gradients in fp32 of a part of the head, trees, odd heads, some sequences idle
        _rotary("rotary_part_f32_back", "f32", 150, 61, 0.8, 2000, 0.7, True, 5, 5, 5, 80, 40, 40, "half", False, 5, True),
        # eight drafts of one conversation: the smallest call there is
        _tree("tree_one_short", "bf16", 1, 8, 0.0, 611, 0.0, False, 0, 32, 8, 128, 16, 3, False),
        # a served batch, sixteen nodes each
        _tree("tree_step_batch", "bf16", 32, 16, 0.3, 8192, 0.7, False, 0, 32, 8, 128, 16, 4, False),
        # wide trees over an 8-bit cache, eight query heads to a key-value head, some sequences idle
        _tree("tree_wide_e4m3", "e4m3", 40, 64, 0.5, 4001, 0.8, True, 2, 64, 8, 128, 64, 8, True),
        # one sequence of two hundred thousand positions: the long axis has to be split
        _tree("tree_long", "bf16", 1, 32, 0.0, 200001, 0.0, False, 0, 32, 8, 128, 64, 4, False),
        # a chain of four drafts of one conversation
        _verify("verify_chain_one", 1, 5, 0.0, False, 0, 32000, "f32", True, 1),
        # trees of sixteen nodes over a wide vocabulary
        _verify("verify_trees", 64, 16, 0.5, False, 0, 131072, "f32", True, 4),
        # drafts without probabilities, an odd vocabulary in bf16, some sequences idle
        _verify("verify_certain_bf16", 200, 7, 0.6, True, 3, 50021, "bf16", False, 2),
        # one layer of a small batch
        _keep("keep_one_layer", "bf16", 1, 16, 8, 0.4, 700, 0.5, 8, 128, 16, False),
        # all 32 layers of a served batch, 8-bit cells
        _keep("keep_layers_e4m3", "e4m3", 32, 64, 24, 0.5, 300, 0.7, 8, 128, 32, True),
    ]


def _rotary(name, *values):
    return _case(name, "rotary", ("dtype", "seqs", "new", "new_spread", "len", "len_spread", "idle", "pad", "heads", "kv", "dim",
                                  "dims", "offset", "layout", "scaled", "branch", "backward"), values)


def _tree(name, *values):
    return _case(name, "tree", ("cache", "seqs", "new", "new_spread", "len", "len_spread", "idle", "pad", "heads", "kv", "dim",
                                "page", "branch", "stats"), values)


def _verify(name, *values):
    c = _case(name, "verify", ("seqs", "new", "new_spread", "idle", "pad", "vocab", "dtype", "drafts", "branch"), values)
    return {**c, "len": c["new"], "len_spread": 0.0}


def _keep(name, *values):
    c = _case(name, "keep", ("cache", "layers", "seqs", "new", "new_spread", "len", "len_spread", "kv", "dim", "page", "idle"),
              values)
    return {**c, "pad": 0}


def _case(name, kind, fields, values):
    c = {"kind": kind, **dict(zip(fields, values, strict=True))}
    return {"name": name, **c} if name else c


def draw(rng):
    """One more case: every size over its range, on a logarithm where the range is wide."""
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def spread():
        return round(rng.uniform(0.0, 0.95), 2)

    kind = rng.choice(("rotary", "tree", "tree", "verify", "keep"))
    idle, pad, kv, fmt = rng.random() < 0.3, rng.choice((0, 0, 1, 6)), rng.choice((1, 2, 4, 5, 8, 12, 16, 32)), rng.choice(("bf16", "e4m3"))
    branch = rng.choice((1, 1, 2, 3, 4, 8, 20))
    if kind == "rotary":
        dims = 2 * rng.randint(4, 64)
        dim = rng.choice((dims, dims + 2 * rng.randint(0, 64), 64 if dims <= 64 else 128))
        new = rng.randint(1, 8) if rng.random() < 0.4 else log(1, 4096)
        c = _rotary(None, rng.choice(("bf16", "f32")), log(1, 200), new, spread(), log(new, 200000), spread(), idle, pad,
                    kv * rng.choice((1, 2, 4, 7)), kv, dim, dims, rng.choice((0, dim - dims)),
                    rng.choice(("half", "interleaved")), rng.random() < 0.5, branch if new <= 128 else 1, rng.random() < 0.2)
    elif kind == "tree":
        new = rng.choice((rng.randint(1, 8), log(1, 128)))
        c = _tree(None, fmt, log(1, 200), new, spread(), log(new, 60000), spread(), idle, pad,
                  kv * rng.choice((1, 1, 2, 3, 4, 5, 7, 8, 16)), kv, rng.choice((64, 128)), rng.choice((16, 32, 64, 128)),
                  branch, rng.random() < 0.4)
    elif kind == "verify":
        c = _verify(None, log(1, 300), rng.choice((rng.randint(1, 8), log(1, 128))), spread(), idle, pad, log(300, 150000),
                    rng.choice(("bf16", "f32")), rng.random() < 0.7, branch)
    else:
        new = log(1, 128)
        c = _keep(None, fmt, log(1, 48), log(1, 100), new, spread(), log(new, 2000), spread(), kv, rng.choice((64, 128)),
                  rng.choice((16, 32, 64, 128)), idle)
    top = max(_cost(x) for x in listed() if x["kind"] == kind)
    least = {"seqs": 4.0, "len": 512.0, "new": 16.0, "layers": 4.0, "vocab": 4000.0}
    while _cost(c) > top or _room(c) > 6e9:
        part = max((k for k in least if k in c and not (kind == "verify" and k == "len")), key=lambda k: c[k] / least[k])
        c[part] = max(1, int(c[part] / rng.uniform(1.2, 2.0)))
        c["new"] = min(c["new"], c["len"]) if kind != "verify" else c["new"]
        c["len"] = c["new"] if kind == "verify" else c["len"]
    return c


# ------------------------------------------------------------------ sizes

def _sizes(c):
    """New rows and lengths of every sequence: spread without chance, so that the case alone says them."""
    new, lens = [], []
    for i in range(c["seqs"]):
        a, b = ((i + 1) * 0.6180339887498949) % 1.0, ((i + 1) * 0.7548776662466927) % 1.0
        n = max(1, round(c["new"] * (1.0 - c["new_spread"] * a)))
        if c["idle"] and i % 5 == 3:
            n = 0
        new.append(n)
        lens.append(max(1, n, round(c["len"] * (1.0 - c["len_spread"] * b))))
    return new, lens


def _parents(c, i, n):
    """Parents of sequence i's nodes: a row back, or up to `branch` rows back."""
    got = [-1]
    for j in range(1, n):
        got.append(j - 1 - int(((j * 0.6180339887498949 + i * 0.7548776662466927) % 1.0) * min(j, c["branch"])))
    return got[:n]


def _depths(parents):
    got = []
    for p in parents:
        got.append(0 if p < 0 else got[p] + 1)
    return got


def _accepted(c, i, n):
    """A branch to keep: some first nodes, then nodes that lie behind all places that are written."""
    count = min(n, 1 + int(((i * 0.5698402909980532 + 0.3) % 1.0) * min(n, 8)))
    same = (count + 1) // 2
    room = n - count
    if room < count - same:
        return list(range(count))
    step = max(1, room // max(1, count - same))
    return list(range(same)) + [count + step * k + (step - 1) // 2 for k in range(count - same)]


def work(c):
    new, lens = _sizes(c)
    table = 4 * (2 * c["seqs"] + 1)
    if c["kind"] == "rotary":
        size = 4 if c["dtype"] == "f32" else 2
        values = sum(new) * (c["heads"] + c["kv"])
        return {"bytes": 2 * values * c["dim"] * size + table + (4 * sum(new) if c["branch"] > 1 else 0), "flops": 3 * values * c["dims"]}
    if c["kind"] == "verify":
        rows = sum(n > 0 for n in new)
        row = c["vocab"] * (4 if c["dtype"] == "f32" else 2)
        drafted = sum(n > 1 for n in new) if c["drafts"] else 0
        return {"bytes": (rows + drafted) * row + 20 * sum(new) + 4 * c["seqs"] * (3 + max(new)) + table, "flops": 3 * (rows + drafted) * c["vocab"]}
    row = c["kv"] * (c["dim"] + 1 if c["cache"] == "e4m3" else 2 * c["dim"])  # one position of K, or of V
    if c["kind"] == "keep":
        moved = sum(sum(p != j for j, p in enumerate(_accepted(c, i, n))) for i, n in enumerate(new))
        return {"bytes": 4 * moved * row * c["layers"] + 4 * c["seqs"] * (2 + max(new)) + table, "flops": 0}
    used = [t for n, t in zip(new, lens) if n]
    pages = sum(-(-t // c["page"]) for t in used)
    pairs = sum(n * (t - n) + sum(_depths(_parents(c, i, n))) + n for i, (n, t) in enumerate(zip(new, lens)))
    rows = sum(new) * c["heads"]
    return {"bytes": 2 * sum(used) * row + rows * (4 * c["dim"] + (8 if c["stats"] else 0)) + table + 4 * pages + 4 * sum(new),
            "flops": 4 * c["dim"] * c["heads"] * pairs}


def _cost(c):
    w = work(c)
    if c["kind"] == "verify":  # what the steps from node to node take
        return c["seqs"] * c["new"] * c["vocab"]
    return max(w["bytes"], w["flops"] / 50)


def _room(c):
    """Bytes of the largest tensor that is made."""
    new, lens = _sizes(c)
    if c["kind"] == "rotary":
        return 8.0 * sum(new) * c["heads"] * c["dim"]
    if c["kind"] == "verify":
        return 4.0 * sum(new) * c["vocab"]
    if c["kind"] == "keep":
        return 2.5 * c["layers"] * sum(-(-t // c["page"]) * c["page"] for t in lens) * c["kv"] * c["dim"]
    return 4.0 * c["seqs"] * max(lens) * max(c["kv"] * c["dim"], c["heads"] * max(new))


# ----------------------------------------------------------------- inputs

_DENSE = {"f32": torch.float32, "bf16": torch.bfloat16}
_THETA, _FACTOR, _ORIGINAL, _LOW, _HIGH = 10000.0, 8.0, 8192, 1.0, 4.0
_FILL = -0.0625  # what outputs hold before a call


def _pack(x):
    """Codes and scale bytes of the last dimension's vectors: 2^k with the least k such that max|x| <= 448 * 2^k."""
    m, e = torch.frexp(x.abs().amax(-1))
    k = torch.where(m > 0, e - 9 + (m > 0.875).to(e.dtype), torch.zeros_like(e)).clamp(-126, 120)
    inverse = ((127 - k) << 23).view(torch.float32)
    return (x * inverse[..., None]).to(torch.float8_e4m3fn), (k + 127).to(torch.uint8)


def _frequencies(c):
    """Radians a position, in 64 bits: those of long wavelengths divided where the context is scaled, blended in between."""
    f = _THETA ** (-torch.arange(0, c["dims"], 2, dtype=torch.float64, device="cuda") / c["dims"])
    if not c["scaled"]:
        return f
    keep = ((_ORIGINAL * f / (2 * math.pi) - _LOW) / (_HIGH - _LOW)).clamp(0.0, 1.0)
    return f * (keep + (1.0 - keep) / _FACTOR)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    new, lens = _sizes(c)
    page = c.get("page", 16)
    most = max(-(-t // page) for t in lens)
    count = sum(-(-t // page) for t in lens)
    pool = count + count // 4 + 2  # a server's pool is never quite full
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    held = torch.tensor([-(-t // page) for t in lens], device="cuda")
    first = torch.cumsum(held, 0) - held
    slot = torch.arange(most, device="cuda")
    named = first[:, None] + slot
    pages = torch.where(slot < held[:, None], order[named.clamp(max=pool - 1)], torch.zeros((), dtype=torch.int32, device="cuda"))
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    rows = starts[-1] + c["pad"]
    s = {"case": c, "rows": starts[-1], "new": max(new), "longest": max(lens), "pages": pages.contiguous(), "starts": ints(starts),
         "lens": ints(lens), "parents": None}
    if c.get("branch", 1) > 1 or c["kind"] == "tree":
        s["parents"] = ints([p for i, n in enumerate(new) for p in _parents(c, i, n)] + [-1] * c["pad"])
    if c["kind"] == "rotary":
        for x, heads in (("q", c["heads"]), ("k", c["kv"])):
            s[x] = normal(rows, heads, c["dim"]).to(_DENSE[c["dtype"]])
            s[x + "_out"] = torch.full_like(s[x], _FILL)
        s["frequencies"] = _frequencies(c)
    elif c["kind"] == "verify":
        _verify_inputs(s, c, new, starts, rows, normal, g)
    else:
        layers = c.get("layers", 1)
        gain = torch.exp(0.4 * normal(c["kv"], 1, c["dim"]))  # keys spread unevenly over their channels
        for x in ("k", "v"):
            cells = torch.empty(layers, pool, c["kv"], page, c["dim"], device="cuda",
                                dtype=torch.float8_e4m3fn if c["cache"] == "e4m3" else torch.bfloat16)
            scale = torch.empty(layers, pool, c["kv"], page, dtype=torch.uint8, device="cuda")
            for layer in range(layers):
                for at in range(0, pool, 4096):  # in pieces, for the fp32 values' room
                    v = normal(min(4096, pool - at), c["kv"], page, c["dim"]) * (gain if x == "k" else 1.0)
                    if c["cache"] == "e4m3":
                        cells[layer, at:at + 4096], scale[layer, at:at + 4096] = _pack(v)
                    else:
                        cells[layer, at:at + 4096] = v.to(torch.bfloat16)
            s[x + "_cache"] = cells
            s[x + "_scale"] = scale if c["cache"] == "e4m3" else None
        if c["kind"] == "tree":
            s["q"] = normal(rows, c["heads"], c["dim"]).to(torch.bfloat16)
            s["out"] = torch.full((rows, c["heads"], c["dim"]), _FILL, dtype=torch.bfloat16, device="cuda")
            s["m"], s["l"] = (torch.full((rows, c["heads"]), _FILL, device="cuda") for _ in range(2))
        else:
            branch = [_accepted(c, i, n) for i, n in enumerate(new)]
            s["path"] = ints([b + [-1] * (max(new) - len(b)) for b in branch])
            s["counts"] = ints([len(b) for b in branch])
            s["lens_out"] = ints([0] * len(new))
    if own:
        _handles(s, c, pool, page)
    return s


def _verify_inputs(s, c, new, starts, rows, normal, g):
    """Target's and draft's probabilities that are alike, and tokens drawn from the draft's at each node's parent."""
    dtype = _DENSE[c["dtype"]]
    s["target"] = torch.empty(rows, c["vocab"], dtype=dtype, device="cuda")
    s["draft"] = torch.empty_like(s["target"]) if c["drafts"] else None
    drawn = torch.empty(rows, dtype=torch.int64, device="cuda")
    for at, (i, n) in zip(starts, enumerate(new)):
        end = at + n if i + 1 < len(new) else rows
        if end == at:
            continue
        logits = 2.5 * normal(end - at, c["vocab"])
        s["target"][at:end] = torch.softmax(logits, -1).to(dtype)
        likely = torch.softmax(logits + 0.7 * normal(end - at, c["vocab"]), -1).to(dtype)
        if c["drafts"]:
            s["draft"][at:end] = likely
        if n > 1:
            up = torch.tensor(_parents(c, i, n)[1:], device="cuda")
            likely = likely.float() if c["drafts"] else likely.float() ** 2  # certain drafts are likely ones
            drawn[at + 1:at + n] = torch.multinomial(likely[up], 1, generator=g)[:, 0]
        drawn[at] = i % c["vocab"]
        drawn[at + n:end] = 0
    s["tokens"] = drawn.to(torch.int32)
    s["accept"] = torch.rand(rows, generator=g, device="cuda")
    s["sample"] = torch.rand(len(new), generator=g, device="cuda")
    s["path"] = torch.zeros(len(new), max(new), dtype=torch.int32, device="cuda")
    s["counts"], s["picked"] = (torch.zeros(len(new), dtype=torch.int32, device="cuda") for _ in range(2))


def _handles(s, c, pool, page):
    """What a user of the framework keeps: relations over the tensors, the batch, the caches, the plan."""
    from tensor_relational_einsum_gb300 import PageBatch, PagedCache, Relation, Rotary
    s["batch"] = PageBatch(s["pages"], s["starts"], s["lens"], max_new=s["new"])
    dense = [x for x in ("q", "k", "q_out", "k_out", "out", "m", "l", "target", "draft") if s.get(x) is not None]
    s["relations"] = {x: Relation("f32" if s[x].dtype == torch.float32 else "bf16", s[x].shape, [1] * s[x].dim(),
                                  storage=s[x].reshape(-1)) for x in dense}
    if c["kind"] == "rotary":
        scaling = {"factor": _FACTOR, "original": _ORIGINAL, "low": _LOW, "high": _HIGH} if c["scaled"] else {}
        s["plan"] = Rotary(c["dims"], theta=_THETA, layout=c["layout"], offset=c["offset"], **scaling)
    elif c["kind"] != "verify":
        def layer(x, n):
            return s[x][n] if s[x] is not None else None

        s["caches"] = [PagedCache(pool, page, c["kv"], c["dim"], c["cache"], k=layer("k_cache", n), v=layer("v_cache", n),
                                  k_scale=layer("k_scale", n), v_scale=layer("v_scale", n)) for n in range(c.get("layers", 1))]


# -------------------------------------------------------------- the passes

def run(s):
    c = s["case"]
    if own:
        return _own(s, c)
    return {"rotary": _rotate, "tree": _attend, "verify": _walk, "keep": _move}[c["kind"]](s, c)


def _held(s):
    """The caches' own buffers: codes as 8-bit floats, scales as powers of two."""
    got = {"k": s["k_cache"], "v": s["v_cache"]}
    if s["k_scale"] is not None:
        got["k_scale"], got["v_scale"] = (s[x + "_scale"].view(torch.float8_e8m0fnu) for x in ("k", "v"))
    return got


def _own(s, c):
    from tensor_relational_einsum_gb300 import cache_attention, cache_keep, rotary, verify_drafts
    r = s["relations"]
    if c["kind"] == "rotary":
        rotary(r["q"], r["k"], s["plan"], s["batch"], parents=s["parents"], q_out=r["q_out"], k_out=r["k_out"], backward=c["backward"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if c["kind"] == "tree":
        cache_attention(r["q"], s["caches"][0], s["batch"], parents=s["parents"], out=r["out"],
                        m_out=r["m"] if c["stats"] else None, l_out=r["l"] if c["stats"] else None)
        return {"out": s["out"], "m": s["m"], "l": s["l"]} if c["stats"] else {"out": s["out"]}
    if c["kind"] == "verify":
        verify_drafts(r["target"], s["batch"], s["tokens"], s["accept"], s["sample"], draft=r.get("draft"), parents=s["parents"],
                      path=s["path"], counts=s["counts"], picked=s["picked"])
        return {"path": s["path"], "counts": s["counts"], "picked": s["picked"]}
    cache_keep(s["caches"], s["batch"], s["path"], s["counts"], lens_out=s["lens_out"])
    return {**_held(s), "lens": s["lens_out"]}


def _ancestors(s):
    """[seq, n, n]: whether node b lies on node a's way to the root, itself included."""
    n = s["new"]
    count = s["starts"][1:] - s["starts"][:-1]
    i = torch.arange(n, device="cuda")
    row = (s["starts"][:-1, None] + i).clamp(max=max(0, s["rows"] - 1)).long()
    up = s["parents"][row] if s["parents"] is not None else (i - 1).expand_as(row)
    a = ((up[..., None] == i) | (i[:, None] == i)).float()
    far = 1
    while far < n:  # ways of twice the length
        a = (torch.matmul(a, a) > 0).float()
        far *= 2
    return (a > 0) & (i < count[:, None])[:, :, None], count, row


def _rotate(s, c):
    r = torch.arange(s["rows"], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["starts"][1:], r, right=True)
    own_row = r - s["starts"][seq]
    at = s["lens"][seq] - (s["starts"][seq + 1] - s["starts"][seq])
    if s["parents"] is None:
        at = at + own_row
    else:
        at = at + _ancestors(s)[0].sum(-1)[seq, own_row.long()] - 1
    angle = at.double()[:, None] * s["frequencies"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if c["backward"]:
        sin = -sin
    half, a, d = c["dims"] // 2, c["offset"], c["dims"]
    for x in ("q", "k"):
        v = s[x][:s["rows"]].float()
        y = v.clone()
        part = slice(a, a + half), slice(a + half, a + d)
        if c["layout"] == "interleaved":
            part = slice(a, a + d, 2), slice(a + 1, a + d, 2)
        y[..., part[0]] = v[..., part[0]] * cos - v[..., part[1]] * sin
        y[..., part[1]] = v[..., part[0]] * sin + v[..., part[1]] * cos
        s[x + "_out"][:s["rows"]] = y.to(s[x].dtype)
    return {"q": s["q_out"], "k": s["k_out"]}


def _cells(s, x, page, slot):
    """Values of cached positions, fp32 [..., heads, dim]."""
    held = s[x + "_cache"][0]
    if s[x + "_scale"] is None:
        return held[page, :, slot].float()
    codes = held.view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn).float()
    return codes * (s[x + "_scale"][0][page, :, slot].to(torch.int32) << 23).view(torch.float32)[..., None]


def _attend(s, c):
    n, t, kv, d = s["new"], s["longest"], c["kv"], c["dim"]
    group = c["heads"] // kv
    anc, count, row = _ancestors(s)
    i, j = torch.arange(n, device="cuda"), torch.arange(t, device="cuda")
    page = s["pages"][:, j // c["page"]].long()                                           # [seq, t]
    slot = (j % c["page"]).expand_as(page)
    q = s["q"][row].float().reshape(-1, n, kv, group, d).permute(0, 2, 3, 1, 4).reshape(-1, kv, group * n, d)
    k = _cells(s, "k", page, slot).permute(0, 2, 3, 1)                                    # [seq, kv, d, t]
    score = torch.matmul(q, k) * (1.0 / math.sqrt(d))
    del q, k
    node = j - (s["lens"] - count)[:, None]                                               # [seq, t]
    see = torch.gather(anc, 2, node.clamp(0, n - 1)[:, None].expand(-1, n, -1))           # [seq, n, t]
    see = ((node < 0)[:, None] | see) & (j < s["lens"][:, None])[:, None]
    see = see[:, None, None]
    score = score.reshape(-1, kv, group, n, t).masked_fill_(~see, -math.inf)
    m = score.amax(-1, keepdim=True)
    p = score.sub_(m.clamp(min=-3.0e38)).exp_()
    total = p.sum(-1, keepdim=True)
    v = _cells(s, "v", page, slot).permute(0, 2, 1, 3)                                    # [seq, kv, t, d]
    o = torch.matmul(p.reshape(-1, kv, group * n, t), v).reshape(-1, kv, group, n, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    kept = i < count[:, None]                                                             # [seq, n]
    rows = row[kept]
    s["out"][rows] = o.permute(0, 3, 1, 2, 4).reshape(-1, n, c["heads"], d)[kept].to(torch.bfloat16)
    if not c["stats"]:
        return {"out": s["out"]}
    s["m"][rows] = m.permute(0, 3, 1, 2, 4).reshape(-1, n, c["heads"])[kept]
    s["l"][rows] = total.permute(0, 3, 1, 2, 4).reshape(-1, n, c["heads"])[kept]
    return {"out": s["out"], "m": s["m"], "l": s["l"]}


def _walk(s, c):
    """Node by node of all sequences together; sums and comparisons in 64 bits, so that no border is crossed by rounding."""
    first, count = s["starts"][:-1].long(), (s["starts"][1:] - s["starts"][:-1]).long()
    last = max(0, s["target"].shape[0] - 1)
    every = torch.arange(c["seqs"], device="cuda")
    at = torch.zeros_like(first)                     # the accepted node
    kept = torch.ones_like(first)
    path = torch.full((c["seqs"], s["new"]), -1, dtype=torch.int64, device="cuda")
    path[:, 0] = 0
    rest = s["target"][first.clamp(max=last)].double()
    mass = torch.ones(c["seqs"], dtype=torch.float64, device="cuda")
    for j in range(1, s["new"]):
        row = (first + j).clamp(max=last)
        up = s["parents"][row].long() if s["parents"] is not None else torch.full_like(row, j - 1)
        asked = (j < count) & (up == at)
        x = s["tokens"][row].long().clamp(0, c["vocab"] - 1)
        if c["drafts"]:
            likely = s["draft"][(first + at).clamp(max=last)].double()
        else:
            likely = torch.zeros_like(rest)
            likely[every, x] = 1.0
        yes = asked & (s["accept"][row].double() * likely[every, x] * mass < rest[every, x])
        no = asked & ~yes
        rest = torch.where(no[:, None], (rest - mass[:, None] * likely).clamp(min=0.0), rest)
        mass = torch.where(no, rest.sum(-1), mass)
        at = torch.where(yes, j, at)
        path.scatter_(1, torch.where(yes, kept, 0)[:, None], torch.where(yes, j, 0)[:, None])
        kept = kept + yes
        rest = torch.where(yes[:, None], s["target"][row].double(), rest)
        mass = torch.where(yes, 1.0, mass)
    rest = torch.where((rest.sum(-1) > 0)[:, None], rest, s["target"][(first + at).clamp(max=last)].double())
    runs = rest.cumsum(-1)
    token = torch.searchsorted(runs, s["sample"].double()[:, None] * runs[:, -1:], right=True)[:, 0].clamp(max=c["vocab"] - 1)
    some = count > 0
    s["path"].copy_(torch.where(some[:, None], path, -1))
    s["counts"].copy_(torch.where(some, kept, 0))
    s["picked"].copy_(torch.where(some & (runs[:, -1] > 0), token, -1))
    return {"path": s["path"], "counts": s["counts"], "picked": s["picked"]}


def _move(s, c):
    base = s["lens"] - (s["starts"][1:] - s["starts"][:-1])
    j = torch.arange(s["path"].shape[1], device="cuda")
    here = j < s["counts"][:, None]
    idle = torch.minimum(base, s["lens"] - 1)[:, None]        # where nothing is kept: a position onto itself
    source, place = (torch.where(here, base[:, None] + x, idle) for x in (s["path"], j))

    def slots(p):
        return torch.gather(s["pages"], 1, torch.div(p, c["page"], rounding_mode="floor").long()).long(), (p % c["page"]).long()

    (from_page, from_slot), (to_page, to_slot) = slots(source), slots(place)
    for x in ("k", "v"):
        cells = s[x + "_cache"]
        raw = cells.view(torch.uint8) if s[x + "_scale"] is not None else cells
        raw[:, to_page, :, to_slot] = raw[:, from_page, :, from_slot]
        if s[x + "_scale"] is not None:
            s[x + "_scale"][:, to_page, :, to_slot] = s[x + "_scale"][:, from_page, :, from_slot]
    s["lens_out"].copy_(base + s["counts"])
    return {**_held(s), "lens": s["lens_out"]}


# ------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """What run() returns, sequence by sequence from the definitions, in 64 bits."""
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    return {"rotary": _exact_rotary, "tree": _exact_tree, "verify": _exact_verify, "keep": _exact_keep}[case["kind"]](s, case)


def _exact_rotary(s, c):
    got = {x: torch.full(s[x].shape, _FILL, dtype=torch.float64, device="cuda") for x in ("q", "k")}
    turn = []
    for i in range(c["dims"] // 2):
        f = math.exp(-2.0 * i / c["dims"] * math.log(_THETA))
        if c["scaled"]:
            wave = 2 * math.pi / f
            if wave > _ORIGINAL / _LOW:
                f /= _FACTOR
            elif wave >= _ORIGINAL / _HIGH:
                w = (_ORIGINAL / wave - _LOW) / (_HIGH - _LOW)
                f = (1.0 - w) * f / _FACTOR + w * f
        turn.append(f)
    turn = torch.tensor(turn, dtype=torch.float64, device="cuda")
    pair = torch.arange(c["dims"] // 2, device="cuda")
    one = c["offset"] + (2 * pair if c["layout"] == "interleaved" else pair)
    two = one + (1 if c["layout"] == "interleaved" else c["dims"] // 2)
    begin = 0
    for i, (n, t) in enumerate(zip(*_sizes(c))):
        if n == 0:
            continue
        deep = list(range(n)) if s["parents"] is None else _depths(_parents(c, i, n))
        angle = (torch.tensor(deep, dtype=torch.float64, device="cuda") + (t - n)).outer(turn)[:, None]
        for x in ("q", "k"):
            z = torch.complex(*(s[x][begin:begin + n][..., w].double() for w in (one, two)))
            z = z * torch.polar(torch.ones_like(angle), -angle if c["backward"] else angle)
            got[x][begin:begin + n] = s[x][begin:begin + n].double()
            got[x][begin:begin + n, :, one], got[x][begin:begin + n, :, two] = z.real, z.imag
        begin += n
    return got


def _exact_tree(s, c):
    got = {"out": torch.full(s["out"].shape, _FILL, dtype=torch.float64, device="cuda")}
    if c["stats"]:
        got["m"], got["l"] = (torch.full(s["m"].shape, _FILL, dtype=torch.float64, device="cuda") for _ in range(2))
    begin = 0
    for i, (n, t) in enumerate(zip(*_sizes(c))):
        if n == 0:
            continue
        drop = torch.zeros(n, t, dtype=torch.float64)
        drop[:, t - n:] = -math.inf
        for a, p in enumerate(_parents(c, i, n)):
            if p >= 0:
                drop[a, t - n:] = drop[p, t - n:]
            drop[a, t - n + a] = 0.0
        drop = drop.cuda()
        whole = s["pages"][i, :-(-t // c["page"])].long()
        kept = {}
        for x in ("k", "v"):
            cells = s[x + "_cache"][0][whole].double()                                    # [pages, kv, page, d]
            if c["cache"] == "e4m3":
                cells = cells * torch.exp2(s[x + "_scale"][0][whole].double() - 127.0)[..., None]
            kept[x] = cells.transpose(0, 1).reshape(c["kv"], -1, c["dim"])[:, :t]
        for h in range(c["heads"]):
            y = h // (c["heads"] // c["kv"])
            a = s["q"][begin:begin + n, h].double() @ kept["k"][y].T / math.sqrt(c["dim"]) + drop
            top = a.max(dim=1).values
            e = torch.exp(a - top[:, None])
            z = e.sum(dim=1)
            got["out"][begin:begin + n, h] = (e @ kept["v"][y]) / z[:, None]
            if c["stats"]:
                got["m"][begin:begin + n, h], got["l"][begin:begin + n, h] = top, z
        begin += n
    return got


def _exact_verify(s, c):
    new, _ = _sizes(c)
    path, counts, picked = [], [], []
    begin = 0
    tokens, accept, sample = (s[x].tolist() for x in ("tokens", "accept", "sample"))
    for i, n in enumerate(new):
        if n == 0:
            path.append([-1] * max(new))
            counts.append(0)
            picked.append(-1)
            continue
        tree, way, v = _parents(c, i, n), [0], 0
        while True:
            r, z = s["target"][begin + v].double(), 1.0
            step = None
            for child in [j for j in range(n) if tree[j] == v]:
                x = tokens[begin + child]
                if c["drafts"]:
                    d = s["draft"][begin + v].double()
                else:
                    d = torch.zeros_like(r)
                    d[x] = 1.0
                if accept[begin + child] * d[x].item() * z < r[x].item():
                    step = child
                    break
                r = torch.clamp(r - z * d, min=0.0)
                z = r.sum().item()
            if step is None:
                break
            way.append(step)
            v = step
        if z == 0.0:
            r = s["target"][begin + v].double()
        sums = torch.cumsum(r, 0)
        picked.append(int((sums <= sample[i] * sums[-1]).sum()) if sums[-1] > 0 else -1)
        path.append(way + [-1] * (max(new) - len(way)))
        counts.append(len(way))
        begin += n
    return {x: torch.tensor(v, dtype=torch.int32, device="cuda") for x, v in (("path", path), ("counts", counts), ("picked", picked))}


def _exact_keep(s, c):
    got = {x: s[x + "_cache"].double() for x in ("k", "v")}
    if c["cache"] == "e4m3":
        got.update({x + "_scale": torch.exp2(s[x + "_scale"].double() - 127.0) for x in ("k", "v")})
    before = {x: v.clone() for x, v in got.items()}
    lens = []
    for i, (n, t) in enumerate(zip(*_sizes(c))):
        branch = _accepted(c, i, n)
        lens.append(t - n + len(branch))
        pages = s["pages"][i].tolist()
        for j, p in enumerate(branch):
            to, source = t - n + j, t - n + p
            if to != source:
                for x in got:
                    got[x][:, pages[to // c["page"]], :, to % c["page"]] = before[x][:, pages[source // c["page"]], :, source % c["page"]]
    got["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return got
