"""The operators of the paged cache, as they are measured: append, read back, attend.

A cache holds the keys and values of many sequences in pages.  A page is
``page`` consecutive positions of one sequence for all key-value heads; a
table names the pages of each sequence in order.  A batch says, for sequence
i, that the rows ``starts[i] .. starts[i + 1]`` of a dense tensor are its last
positions, the sequence being ``lens[i]`` positions long.

* append   new rows of K and V into their pages; an "e4m3" cache holds 8-bit
           codes and one power-of-two scale per position and head:
           2^k with the least k such that max|x| <= 448 * 2^k;
* read     the positions of the batch out of their pages into dense rows;
* attend   softmax attention of the batch's query rows over their sequences'
           pages, query heads in groups that share a key-value head.

``run`` computes them in elementary torch operations, or, where ``own`` is
true, calls the framework's operators.
"""
import math

import torch

own = False

_FIELDS = ("kind", "cache", "seqs", "new", "new_spread", "len", "len_spread", "idle", "pad", "heads", "kv", "dim", "page",
           "dense", "causal", "stats")


def _case(name, *values):
    c = dict(zip(_FIELDS, values))
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decoding step of a small batch writes one position per sequence: latency alone
        _case("append_step", "append", "bf16", 32, 1, 0.0, 2048, 0.8, False, 0, 8, 8, 128, 16, "bf16", True, False),
        # prompts of four sequences enter an 8-bit cache, all 32 heads kept
        _case("append_prompts_e4m3", "append", "e4m3", 4, 4096, 0.5, 6000, 0.3, False, 3, 32, 32, 128, 64, "bf16", True,
              False),
        # ragged small chunks in fp32, some sequences idle, an odd head count
        _case("append_ragged_f32_e4m3", "append", "e4m3", 23, 37, 0.9, 911, 0.7, True, 5, 5, 5, 64, 32, "f32", True, False),
        # whole sequences leave the cache for the dense path (prefix re-use, offload)
        _case("read_whole_bf16", "read", "bf16", 8, 8192, 0.2, 8192, 0.2, False, 0, 8, 8, 128, 16, "bf16", True, False),
        # short ragged pieces of an 8-bit cache back to fp32
        _case("read_ragged_e4m3_f32", "read", "e4m3", 48, 700, 0.9, 1500, 0.8, True, 7, 4, 4, 64, 32, "f32", True, False),
        # the first tokens of one conversation: the smallest call there is
        _case("attend_one_short", "attend", "bf16", 1, 1, 0.0, 97, 0.0, False, 0, 32, 8, 128, 16, "bf16", True, False),
        # one decoding step of a served batch with lengths spread widely
        _case("attend_step_batch", "attend", "bf16", 64, 1, 0.0, 8192, 0.7, False, 0, 32, 8, 128, 16, "bf16", True, False),
        # the same over an 8-bit cache, eight query heads to a key-value head, some sequences idle
        _case("attend_step_e4m3", "attend", "e4m3", 160, 1, 0.0, 4001, 0.8, True, 2, 64, 8, 128, 64, "bf16", True, True),
        # one sequence of two hundred thousand positions: the long axis has to be split
        _case("attend_step_long", "attend", "bf16", 1, 1, 0.0, 200001, 0.0, False, 0, 32, 8, 128, 64, "bf16", True, False),
        # a few query rows over an encoder's stored keys, three heads to a group
        _case("attend_cross_ragged", "attend", "bf16", 24, 33, 0.9, 1500, 0.6, False, 4, 15, 5, 64, 32, "bf16", False, True),
        # a chunk of a long prompt over what an 8-bit cache holds of it already
        _case("attend_chunk_e4m3", "attend", "e4m3", 2, 640, 0.4, 9001, 0.3, False, 0, 32, 8, 128, 16, "bf16", True, False),
        # prompts from their first position, 32 heads of 128, nothing cached before
        _case("attend_prompts", "attend", "bf16", 4, 2048, 0.3, 2048, 0.3, False, 0, 32, 32, 128, 128, "bf16", True, False),
    ]


def draw(rng):
    """One more case: every size over its range, on a logarithm where the range is wide."""
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    top = max(_cost(c) for c in listed())
    kind = rng.choice(("append", "read", "attend", "attend"))
    kv = rng.choice((1, 2, 4, 5, 8, 12, 16, 32))
    group = rng.choice((1, 1, 2, 3, 4, 5, 7, 8, 16)) if kind == "attend" else 1
    step = kind == "attend" and rng.random() < 0.5
    c = _case(None, kind, rng.choice(("bf16", "e4m3")), log(1, 200), rng.randint(1, 4) if step else log(1, 4096),
              round(rng.uniform(0.0, 0.95), 2), log(1, 60000), round(rng.uniform(0.0, 0.95), 2), rng.random() < 0.3,
              rng.choice((0, 0, 1, 6)), kv * group, kv, rng.choice((64, 128)), rng.choice((16, 32, 64, 128)),
              "bf16" if kind == "attend" else rng.choice(("bf16", "f32")), kind != "attend" or rng.random() < 0.8,
              kind == "attend" and rng.random() < 0.4)
    if c["causal"]:
        c["len"] = max(c["len"], c["new"])
    while _cost(c) > top or _room(c) > 6e9:
        part = max(("seqs", "len", "new"), key=lambda k: c[k] / {"seqs": 4.0, "len": 512.0, "new": 64.0}[k])
        c[part] = max(1, int(c[part] / rng.uniform(1.2, 2.0)))
        if c["causal"]:
            c["new"] = min(c["new"], c["len"])
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
        t = max(1, round(c["len"] * (1.0 - c["len_spread"] * b)))
        new.append(n)
        lens.append(max(t, n) if c["causal"] else t)
    return new, lens


def _pairs(c, n, t):
    """Kept (query, key) pairs of a sequence."""
    return n * (t - n) + n * (n + 1) // 2 if c["causal"] else n * t


def work(c):
    new, lens = _sizes(c)
    cell = 1 if c["cache"] == "e4m3" else 2
    row = c["kv"] * (c["dim"] * cell + (1 if c["cache"] == "e4m3" else 0))  # one position of K, or of V
    dense = 4 if c["dense"] == "f32" else 2
    table = 4 * (2 * c["seqs"] + 1)
    if c["kind"] != "attend":
        pages = sum((t - 1) // c["page"] - (t - n) // c["page"] + 1 for n, t in zip(new, lens) if n)
        return {"bytes": 2 * sum(new) * (row + c["kv"] * c["dim"] * dense) + table + 4 * pages, "flops": 0}
    used = [t for n, t in zip(new, lens) if n]
    pages = sum(-(-t // c["page"]) for t in used)
    rows = sum(new) * c["heads"]
    return {"bytes": 2 * sum(used) * row + rows * (4 * c["dim"] + (8 if c["stats"] else 0)) + table + 4 * pages,
            "flops": 4 * c["dim"] * c["heads"] * sum(_pairs(c, n, t) for n, t in zip(new, lens))}


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


def _room(c):
    """Bytes of the largest tensor that the plain form makes."""
    new, lens = _sizes(c)
    if c["kind"] != "attend":
        return 4.0 * max(sum(new), sum(lens)) * c["kv"] * c["dim"]
    return 4.0 * c["seqs"] * max(lens) * max(c["kv"] * c["dim"], c["heads"] * max(new))


# ----------------------------------------------------------------- inputs

_DENSE = {"f32": torch.float32, "bf16": torch.bfloat16}


def _pack(x):
    """Codes and scale bytes of the last dimension's vectors: 2^k with the least k such that max|x| <= 448 * 2^k."""
    m, e = torch.frexp(x.abs().amax(-1))
    k = torch.where(m > 0, e - 9 + (m > 0.875).to(e.dtype), torch.zeros_like(e)).clamp(-126, 120)
    inverse = ((127 - k) << 23).view(torch.float32)
    return (x * inverse[..., None]).to(torch.float8_e4m3fn), (k + 127).to(torch.uint8)


def _scale(byte):
    """2^k of the scale bytes (k >= -126)."""
    return (byte.to(torch.int32) << 23).view(torch.float32)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    new, lens = _sizes(c)
    most = max(-(-t // c["page"]) for t in lens)
    count = sum(-(-t // c["page"]) for t in lens)
    pool = count + count // 4 + 2  # a server's pool is never quite full
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    held = torch.tensor([-(-t // c["page"]) for t in lens], device="cuda")
    first = torch.cumsum(held, 0) - held
    slot = torch.arange(most, device="cuda")
    named = first[:, None] + slot
    pages = torch.where(slot < held[:, None], order[named.clamp(max=pool - 1)], torch.zeros((), dtype=torch.int32, device="cuda"))
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s = {"case": c, "rows": starts[-1], "new": max(new), "longest": max(lens),
         "pages": pages.contiguous(), "starts": torch.tensor(starts, dtype=torch.int32, device="cuda"),
         "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    gain = torch.exp(0.4 * normal(c["kv"], 1, c["dim"]))  # keys spread unevenly over their channels
    for x in ("k", "v"):
        held_in = torch.empty(pool, c["kv"], c["page"], c["dim"], device="cuda",
                              dtype=torch.float8_e4m3fn if c["cache"] == "e4m3" else torch.bfloat16)
        scale = torch.empty(pool, c["kv"], c["page"], dtype=torch.uint8, device="cuda")
        for at in range(0, pool, 4096):  # in pieces, for the fp32 values' room
            v = normal(min(4096, pool - at), c["kv"], c["page"], c["dim"]) * (gain if x == "k" else 1.0)
            if c["cache"] == "e4m3":
                held_in[at:at + 4096], scale[at:at + 4096] = _pack(v)
            else:
                held_in[at:at + 4096] = v.to(torch.bfloat16)
        s[x + "_cache"] = held_in
        s[x + "_scale"] = scale if c["cache"] == "e4m3" else None
    rows = starts[-1] + c["pad"]
    if c["kind"] == "append":
        for x in ("k", "v"):
            s[x] = (normal(rows, c["kv"], c["dim"]) * (gain[:, 0] if x == "k" else 1.0)).to(_DENSE[c["dense"]])
    elif c["kind"] == "read":
        for x in ("k", "v"):
            s[x] = torch.full((rows, c["kv"], c["dim"]), -0.0625, dtype=_DENSE[c["dense"]], device="cuda")
    else:
        s["q"] = normal(rows, c["heads"], c["dim"]).to(torch.bfloat16)
        s["out"] = torch.full((rows, c["heads"], c["dim"]), -0.0625, dtype=torch.bfloat16, device="cuda")
        s["m"], s["l"] = (torch.full((rows, c["heads"]), -0.0625, device="cuda") for _ in range(2))
    if own:
        from tensor_relational_einsum_gb300 import PageBatch, PagedCache, Relation

        def relation(t):
            return Relation("f32" if t.dtype == torch.float32 else "bf16", t.shape, [1] * t.dim(), storage=t.reshape(-1))

        s["cache"] = PagedCache(pool, c["page"], c["kv"], c["dim"], c["cache"], k=s["k_cache"], v=s["v_cache"],
                                k_scale=s["k_scale"], v_scale=s["v_scale"])
        s["batch"] = PageBatch(s["pages"], s["starts"], s["lens"], max_new=max(new))
        s["relations"] = {x: relation(s[x]) for x in ("k", "v", "q", "out", "m", "l") if x in s}
    return s


# -------------------------------------------------------------- the passes

def run(s):
    c = s["case"]
    if own:
        return _own(s, c)
    if c["kind"] == "append":
        return _append(s, c)
    return _read(s, c) if c["kind"] == "read" else _attend(s, c)


def _held(s):
    """The cache's own buffers: codes as 8-bit floats, scales as powers of two."""
    got = {"k": s["k_cache"], "v": s["v_cache"]}
    if s["k_scale"] is not None:
        got["k_scale"], got["v_scale"] = (s[x + "_scale"].view(torch.float8_e8m0fnu) for x in ("k", "v"))
    return got


def _own(s, c):
    from tensor_relational_einsum_gb300 import cache_append, cache_attention, cache_read
    r = s["relations"]
    if c["kind"] == "append":
        cache_append(s["cache"], s["batch"], r["k"], r["v"])
        return _held(s)
    if c["kind"] == "read":
        cache_read(s["cache"], s["batch"], k=r["k"], v=r["v"])
        return {"k": s["k"], "v": s["v"]}
    cache_attention(r["q"], s["cache"], s["batch"], causal=c["causal"], out=r["out"],
                    m_out=r["m"] if c["stats"] else None, l_out=r["l"] if c["stats"] else None)
    return {"out": s["out"], "m": s["m"], "l": s["l"]} if c["stats"] else {"out": s["out"]}


def _places(s, c):
    """Page and slot of every row of the batch."""
    row = torch.arange(s["rows"], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["starts"][1:], row, right=True)
    position = s["lens"][seq] - s["starts"][seq + 1] + row
    return s["pages"][seq, position // c["page"]].long(), (position % c["page"]).long()


def _append(s, c):
    page, slot = _places(s, c)
    for x in ("k", "v"):
        values, held = s[x][:s["rows"]].float(), s[x + "_cache"]
        if c["cache"] == "e4m3":
            codes, scale = _pack(values)
            held.view(torch.uint8)[page, :, slot] = codes.view(torch.uint8)
            s[x + "_scale"][page, :, slot] = scale
        else:
            held[page, :, slot] = values.to(torch.bfloat16)
    return _held(s)


def _cells(s, x, page, slot):
    """Values of cached positions, fp32 [..., heads, dim]."""
    held = s[x + "_cache"]
    if s[x + "_scale"] is None:
        return held[page, :, slot].float()
    codes = held.view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn).float()
    return codes * _scale(s[x + "_scale"][page, :, slot])[..., None]


def _read(s, c):
    page, slot = _places(s, c)
    for x in ("k", "v"):
        s[x][:s["rows"]] = _cells(s, x, page, slot).to(s[x].dtype)
    return {"k": s["k"], "v": s["v"]}


def _attend(s, c):
    n, t, kv, d = s["new"], s["longest"], c["kv"], c["dim"]
    group = c["heads"] // kv
    count = s["starts"][1:] - s["starts"][:-1]
    i, j = torch.arange(n, device="cuda"), torch.arange(t, device="cuda")
    row = (s["starts"][:-1, None] + i).clamp(max=s["q"].shape[0] - 1).long()             # [seq, n]
    page = s["pages"][:, j // c["page"]].long()                                           # [seq, t]
    slot = (j % c["page"]).expand_as(page)
    q = s["q"][row].float().reshape(-1, n, kv, group, d).permute(0, 2, 3, 1, 4).reshape(-1, kv, group * n, d)
    k = _cells(s, "k", page, slot).permute(0, 2, 3, 1)                                    # [seq, kv, d, t]
    score = torch.matmul(q, k) * (1.0 / math.sqrt(d))
    del q, k
    see = (j < s["lens"][:, None])[:, None, :]                                            # [seq, 1, t]
    if c["causal"]:
        see = see & (j <= (s["lens"] - count)[:, None, None] + i[:, None])               # [seq, n, t]
    see = see.expand(-1, n, t)[:, None, None]
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


# ------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """What run() returns, sequence by sequence from the definitions, in 64 bits."""
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    c, page, kinds = case, case["page"], ("k", "v")
    begin = 0
    if c["kind"] == "append":
        got = {x: s[x + "_cache"].double() for x in kinds}
        if c["cache"] == "e4m3":
            got.update({x + "_scale": torch.exp2(s[x + "_scale"].double() - 127.0) for x in kinds})
    elif c["kind"] == "read":
        got = {x: torch.full(s[x].shape, -0.0625, dtype=torch.float64, device="cuda") for x in kinds}
    else:
        got = {"out": torch.full(s["out"].shape, -0.0625, dtype=torch.float64, device="cuda")}
        if c["stats"]:
            got["m"], got["l"] = (torch.full(s["m"].shape, -0.0625, dtype=torch.float64, device="cuda") for _ in range(2))
    for i, (n, t) in enumerate(zip(*_sizes(c))):
        end = begin + n
        if n == 0:
            continue
        if c["kind"] == "append":
            for x in kinds:
                value = s[x][begin:end].double()
                where = torch.arange(t - n, t, device="cuda")
                at = (s["pages"][i].long()[torch.div(where, page, rounding_mode="floor")], slice(None), where.remainder(page))
                if c["cache"] == "e4m3":
                    largest = value.abs().max(dim=-1).values
                    power = torch.exp2(torch.where(largest > 0, torch.ceil(torch.log2(largest / 448.0) - 1e-10), largest))
                    got[x + "_scale"][at] = power
                    value = value / power[:, :, None]
                got[x][at] = value
        else:
            whole = s["pages"][i, :-(-t // page)].long()
            kept = {}
            for x in kinds:
                cells = s[x + "_cache"][whole].double()                                  # [pages, kv, page, d]
                if c["cache"] == "e4m3":
                    cells = cells * torch.exp2(s[x + "_scale"][whole].double() - 127.0)[..., None]
                kept[x] = cells.transpose(0, 1).reshape(c["kv"], -1, c["dim"])[:, :t]
            if c["kind"] == "read":
                for x in kinds:
                    got[x][begin:end] = kept[x][:, t - n:].transpose(0, 1)
            else:
                for h in range(c["heads"]):
                    y = h // (c["heads"] // c["kv"])
                    a = s["q"][begin:end, h].double() @ kept["k"][y].T / math.sqrt(c["dim"])
                    if c["causal"]:
                        a += torch.full_like(a, -math.inf).triu(t - n + 1)
                    top = a.max(dim=1).values
                    e = torch.exp(a - top[:, None])
                    z = e.sum(dim=1)
                    got["out"][begin:end, h] = (e @ kept["v"][y]) / z[:, None]
                    if c["stats"]:
                        got["m"][begin:end, h], got["l"][begin:end, h] = top, z
        begin = end
    return got
