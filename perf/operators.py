"""The serving operators of a drafting round, as they are measured.

    attend   attention of R query rows a sequence over context caches held in four bits
    write    rows of keys and values quantised into such a cache, and read back as the values they stand for
    select   the selector's chain with every token sampled from its row's candidates
    verify   drafted tokens verified against the target's probabilities

``run`` takes the plain forms (elementary torch operations) where ``own`` is false, and the library's
operators where it is true, on the same state.
"""
import torch

own = False

TILE = 128          # cache rows of one tile of a four-bit cache
GROUP = 32          # values that share a scale
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one token of 32 sequences decoded over 8,192 rows each: the large serving step
        dict(name="attend-token-32", op="attend", batch=32, rows=1, heads=32, kv=8, hd=128, length=8192, step=37,
             window=0, causal=True, dtype="bf16"),
        # one token of one short sequence: launches and latency
        dict(name="attend-token-1", op="attend", batch=1, rows=1, heads=4, kv=2, hd=64, length=333, step=0,
             window=0, causal=True, dtype="f32"),
        # the drafter's own block over the longest context of its workloads
        dict(name="attend-block-32k", op="attend", batch=1, rows=16, heads=32, kv=8, hd=128, length=32768, step=0,
             window=0, causal=False, dtype="f32"),
        # 32 blocks over 8,192 rows each (the batched workload), ragged
        dict(name="attend-block-32", op="attend", batch=32, rows=16, heads=16, kv=8, hd=128, length=8192, step=61,
             window=0, causal=False, dtype="f32"),
        # a target's check of 9 drafted rows, causal within a sliding window, ranges that start inside a tile
        dict(name="attend-window-8", op="attend", batch=8, rows=9, heads=32, kv=8, hd=128, length=6001, step=129,
             window=2048, causal=True, dtype="f16"),
        # a prompt's rows into the cache, the largest write
        dict(name="write-prompt", op="write", batch=8, n=4096, kv=8, hd=128, at=77, dtype="bf16"),
        # one decoded token of 32 sequences
        dict(name="write-token", op="write", batch=32, n=1, kv=8, hd=128, at=4095, dtype="f32"),
        # one sequence's draft at the full vocabulary
        dict(name="select-1", op="select", batch=1, k=15, width=151936, vocab=151936, rank=64, top=16),
        # 32 sequences
        dict(name="select-32", op="select", batch=32, k=15, width=151936, vocab=151936, rank=64, top=16),
        # one sequence's greedy draft (every proposal certain), the smallest vocabulary
        dict(name="verify-small", op="verify", batch=2, k=4, vocab=4096, top=0, dtype="f16", ragged=False),
        # one sequence's sampled draft at the full vocabulary
        dict(name="verify-1", op="verify", batch=1, k=15, vocab=151936, top=16, dtype="f32", ragged=False),
        # 32 sequences, drafts of different lengths, some sequences greedy
        dict(name="verify-32", op="verify", batch=32, k=15, vocab=151936, top=16, dtype="bf16", ragged=True),
    ]


def _log(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "write", "select", "verify", "verify"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "attend":
        hd, kv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
        rows = rng.choice([1, 1, rng.randint(2, 16), 16])
        rep = rng.choice([r for r in (1, 2, 3, 4, 6, 8) if r * rows <= 64])
        batch = _log(rng, 1, 32)
        most = min(1, 32 / (rep * rows)) * 32 * 8192 * 8 / (batch * kv)
        length = _log(rng, 1, min(65536, int(most)))
        return dict(op=op, batch=batch, rows=rows, heads=kv * rep, kv=kv, hd=hd, length=length,
                    step=rng.randint(0, max(0, length // batch - 1)), window=rng.choice([0, 0, _log(rng, 1, 4096)]),
                    causal=rng.random() < 0.5, dtype=dtype)
    if op == "write":
        batch = _log(rng, 1, 32)
        return dict(op=op, batch=batch, n=_log(rng, 1, 32768 // batch), kv=rng.choice([1, 2, 4, 8]),
                    hd=rng.choice([64, 128]), at=rng.randint(0, 300), dtype=dtype)
    if op == "select":
        vocab = 16 * _log(rng, 64, 9496)
        return dict(op=op, batch=_log(rng, 1, 32), k=rng.randint(1, 15), width=rng.randint(vocab // 2, vocab),
                    vocab=vocab, rank=rng.choice([16, 64, 128]), top=rng.choice([1, 4, 8, 16, 32]))
    return dict(op=op, batch=_log(rng, 1, 32), k=rng.randint(0, 15), vocab=_log(rng, 1000, 151936),
                top=rng.choice([0, 1, 8, 16, 32]), dtype=dtype, ragged=rng.random() < 0.5)


# ---------------------------------------------------------------------------------- sizes that follow from a case

def _ranges(c):
    """Per sequence the cache rows [lo, hi) that are read and the row of its first query."""
    n = [max(1, c["length"] - b * c["step"]) for b in range(c["batch"])]
    anchor = [max(0, x - c["rows"]) if c["causal"] else x for x in n]
    lo = [max(0, a + 1 - c["window"]) if c["window"] else 0 for a in anchor]
    return [min(l, x) for l, x in zip(lo, n)], n, anchor


def _drafted(c):
    return [c["k"] - b % (c["k"] + 1) if c["ragged"] and b % 3 else c["k"] for b in range(c["batch"])]


def work(case):
    c = case
    if c["op"] == "attend":
        lo, hi, _ = _ranges(c)
        n = sum(h - l for l, h in zip(lo, hi))
        q = c["batch"] * c["rows"] * c["heads"] * c["hd"]
        return {"bytes": 2 * n * c["kv"] * (c["hd"] // 2 + c["hd"] // 16) + 2 * q * SIZE[c["dtype"]],
                "flops": 4 * n * c["rows"] * c["heads"] * c["hd"]}
    if c["op"] == "write":
        x = 2 * c["batch"] * c["n"] * c["kv"] * c["hd"]
        # the rows in, the four-bit rows out, and read back as f32
        return {"bytes": x * SIZE[c["dtype"]] + 2 * (x // 2 + x // 16) + 4 * x, "flops": 4 * x}
    if c["op"] == "select":
        rows = c["batch"] * c["k"]
        books = rows * (c["top"] + 1) * c["rank"] * 2           # a predecessor's row, the candidates' rows
        return {"bytes": rows * (c["width"] * 4 + c["rank"] * 4 + c["top"] * 8 + 8) + books,
                "flops": rows * (c["width"] + 3 * c["top"] * c["rank"])}
    rows = sum(d + 1 for d in _drafted(c))
    return {"bytes": rows * (c["vocab"] * SIZE[c["dtype"]] + 8 * c["top"] + 16), "flops": rows * c["vocab"] * 4}


# ---------------------------------------------------------------------------------- the four-bit cache in torch

def _order(device):
    """Place (byte, high nibble) of each of the 8 values of a 32-bit word, as an index into its 8 nibbles: a word
    holds values 0 2 4 6 in its low half and 1 3 5 7 in its high half, lowest nibble first."""
    return torch.tensor([0, 4, 1, 5, 2, 6, 3, 7], device=device)


def _quantise(x):
    """Codes (-7..7) and scales of x [..., hd] (f32), one scale for each 32 values."""
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    scale = (g.abs().amax(-1) / 7).to(torch.bfloat16).to(torch.float16)
    s = scale.float().unsqueeze(-1)
    q = torch.where(s > 0, torch.round(g / torch.where(s > 0, s, 1)), torch.zeros_like(g)).clamp(-7, 7)
    return q, scale


def _pack(x):
    """x f32 [B][rows][kv][hd], rows a multiple of 128, as the cache's bytes [B][kv][rows / 128][tile]."""
    B, n, kv, hd = x.shape
    q, scale = _quantise(x.permute(0, 2, 1, 3).reshape(B, kv, n // TILE, TILE, hd))
    u = (q + 8).to(torch.uint8).reshape(B, kv, n // TILE, TILE, hd // GROUP, 4, 8)
    words = torch.empty_like(u)
    words[..., _order(x.device)] = u
    code = (words[..., 0::2] | (words[..., 1::2] << 4)).reshape(B, kv, n // TILE, TILE, hd // GROUP, 16)
    code = code.transpose(3, 4).reshape(B, kv, n // TILE, -1)
    return torch.cat([code, scale.contiguous().view(torch.uint8).reshape(B, kv, n // TILE, -1)], -1).contiguous()


def _unpack(buf, hd):
    """The values that a cache's bytes stand for, f32 [B][kv][rows][hd]."""
    B, kv, t = buf.shape[:3]
    G = hd // GROUP
    code = buf[..., :TILE * hd // 2].reshape(B, kv, t, G, TILE, 16).transpose(3, 4)
    nib = torch.stack([code & 15, code >> 4], -1).reshape(B, kv, t, TILE, G, 4, 8)
    q = nib[..., _order(buf.device)].float() - 8
    scale = buf[..., TILE * hd // 2:].contiguous().view(torch.float16).reshape(B, kv, t, TILE, G, 1).float()
    return (q.reshape(B, kv, t, TILE, G, GROUP) * scale).reshape(B, kv, t * TILE, hd)


# ---------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _prepare_attend(c, seed):
    g = _gen(seed)
    lo, hi, anchor = _ranges(c)
    tiles = (max(hi) + TILE - 1) // TILE
    shape = (1, tiles * TILE, c["kv"], c["hd"])
    ks, vs = [], []
    for b in range(c["batch"]):
        # keys as a norm leaves them, some channels larger than the rest; values around one
        k = torch.randn(shape, generator=g, device="cuda") * (1 + 2 * torch.rand(c["kv"], c["hd"], generator=g,
                                                                                  device="cuda") ** 4)
        v = torch.randn(shape, generator=g, device="cuda")
        k, v = _pack(k), _pack(v)
        # rows outside a sequence's range hold whatever was there before, scales that are not numbers among it
        for t in (k, v):
            scale = t[..., TILE * c["hd"] // 2:].contiguous().view(torch.int16).reshape(1, c["kv"], tiles * TILE, -1)
            scale[:, :, hi[b]:] = 0x7E00
            scale[:, :, :lo[b]] = 0x7E00
            t[..., TILE * c["hd"] // 2:] = scale.reshape(1, c["kv"], tiles, -1).view(torch.uint8)
        ks.append(k)
        vs.append(v)
    q = torch.randn(c["batch"], c["rows"], c["heads"], c["hd"], generator=g, device="cuda").to(TYPES[c["dtype"]])
    st = dict(c=c, q=q, k=torch.cat(ks), v=torch.cat(vs), lo=lo, hi=hi, anchor=anchor)
    st["range"] = [torch.tensor(x, device="cuda").view(-1, 1, 1) for x in (lo, hi, anchor)]
    return st


def _prepare_write(c, seed):
    g = _gen(seed)
    shape = (c["batch"], c["n"], c["kv"], c["hd"])
    k = torch.randn(shape, generator=g, device="cuda") * 2
    v = torch.randn(shape, generator=g, device="cuda")
    v[:, ::5, :, :GROUP] = 0                  # a group of zeros
    tiles = (c["at"] + c["n"] + TILE - 1) // TILE
    size = (c["batch"], c["kv"], tiles, TILE * (c["hd"] // 2 + c["hd"] // 16))
    t = TYPES[c["dtype"]]
    return dict(c=c, k=k.to(t), v=v.to(t), at=[c["at"]] * c["batch"],
                ck=torch.zeros(size, dtype=torch.uint8, device="cuda"),
                cv=torch.zeros(size, dtype=torch.uint8, device="cuda"))


def _prepare_select(c, seed):
    g = _gen(seed)
    b, k = c["batch"], c["k"]
    book = lambda: (torch.randn(c["vocab"], c["rank"], generator=g, device="cuda") / c["rank"] ** 0.5).half()  # noqa: E731
    st = dict(c=c, pred=book(), succ=book(),
              logits=torch.randn(b, k, c["width"], generator=g, device="cuda") * 2,
              hp=torch.randn(b, k, c["rank"], generator=g, device="cuda"),
              anchor=torch.randint(0, c["vocab"], (b,), generator=g, device="cuda", dtype=torch.int32),
              u=torch.rand(b, k, generator=g, device="cuda"),
              temperature=0.5 + torch.rand(b, generator=g, device="cuda"))
    st["temperature"][2::4] = 0               # every fourth sequence greedy
    return st


def _prepare_verify(c, seed):
    g = _gen(seed)
    b, k, v = c["batch"], c["k"], c["vocab"]
    # a target's logits: a wide floor and a few tokens well above it
    x = torch.randn(b, k + 1, v, generator=g, device="cuda") * 1.5
    peak = torch.randint(0, v, (b, k + 1, 8), generator=g, device="cuda")
    x.scatter_(2, peak, 9 + 4 * torch.rand(b, k + 1, 8, generator=g, device="cuda"))
    x[:, :, 5::97] = float("-inf")            # tokens that a grammar forbids
    st = dict(c=c, logits=x.to(TYPES[c["dtype"]]), u=torch.rand(b, k + 1, generator=g, device="cuda"),
              temperature=0.6 + 0.8 * torch.rand(b, generator=g, device="cuda"), cand=None, q=None, n=None)
    st["temperature"][3::4] = 0               # every fourth sequence greedy
    if c["top"]:
        cand = torch.rand(b, k, v, generator=g, device="cuda").topk(c["top"], -1).indices
        m = min(c["top"], 8)
        cand[..., :m] = peak[:, :k, :m]       # the drafter mostly knows the target's favourites
        st["cand"] = cand.int()
        w = torch.randn(b, k, c["top"], generator=g, device="cuda") + 2 * (torch.arange(c["top"], device="cuda") < m)
        st["q"] = torch.softmax(w, -1)
        at = torch.multinomial(st["q"].reshape(-1, c["top"]), 1, generator=g).reshape(b, k, 1) if k else \
            torch.zeros(b, 0, 1, dtype=torch.int64, device="cuda")
        st["drafted"] = st["cand"].gather(2, at).squeeze(2).contiguous()
    else:
        st["drafted"] = x[:, :k].argmax(-1).int()
        st["drafted"][:, 2::5] = peak[:, 2:k:5, 0].int()
    if c["ragged"]:
        st["n"] = torch.tensor(_drafted(c), dtype=torch.int32, device="cuda")
    return st


def prepare(case, seed):
    return globals()["_prepare_" + case["op"]](case, seed)


# ---------------------------------------------------------------------------------- the plain forms

def _plain_attend(st):
    c, q = st["c"], st["q"].float()
    lo, hi, anchor = st["range"]
    B, R, H, hd = q.shape
    k, v = _unpack(st["k"], hd), _unpack(st["v"], hd)
    n = k.shape[2]
    row, r = torch.arange(n, device="cuda").view(1, 1, n), torch.arange(R, device="cuda").view(1, R, 1)
    see = ((row >= lo) & (row < hi)).expand(B, R, n)
    if c["window"]:
        see = see & (row >= anchor + r + 1 - c["window"])
    if c["causal"]:
        see = see & (row <= anchor + r)
    held = ((row >= lo) & (row < hi)).view(B, 1, n, 1)
    k, v = torch.where(held, k, 0.0), torch.where(held, v, 0.0)
    qg = q.view(B, R, c["kv"], -1, hd).permute(0, 2, 3, 1, 4).reshape(B, c["kv"], -1, hd)      # [B][kv][rep * R][hd]
    s = (qg @ k.transpose(2, 3)).view(B, c["kv"], -1, R, n) * hd ** -0.5
    s = s.masked_fill(~see.view(B, 1, 1, R, n), float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == float("-inf"), 0.0, m))
    l = p.sum(-1, keepdim=True)
    y = (p.reshape(B, c["kv"], -1, n) @ v).view(B, c["kv"], -1, R, hd)
    y = torch.where(l > 0, y / l, 0.0)
    return y.permute(0, 3, 1, 2, 4).reshape(B, R, H, hd).to(st["q"].dtype)


def _plain_write(st):
    out = []
    for x in (st["k"].float(), st["v"].float()):
        q, s = _quantise(x)
        out.append((q * s.float().unsqueeze(-1)).reshape(x.shape))
    return tuple(out)


def _first_largest(x):
    """The lowest index of the largest value of the last dimension, which is kept."""
    i = torch.arange(x.shape[-1], device=x.device)
    return torch.where(x == x.amax(-1, keepdim=True), i, x.shape[-1] - 1).amin(-1, keepdim=True)


def _plain_select(st):
    c, T = st["c"], st["temperature"].double().view(-1, 1)
    top, b = c["top"], c["batch"]
    value, index = torch.sort(st["logits"], dim=-1, descending=True, stable=True)
    value, index = value[..., :top].double(), index[..., :top]
    prev = st["anchor"].long()
    chosen, probs = [], []
    for j in range(c["k"]):
        pred = st["pred"][prev].double() * st["hp"][:, j].double()
        s = value[:, j] + (st["succ"][index[:, j]].double() * pred.unsqueeze(1)).sum(-1)
        w = torch.exp((s - s.amax(-1, keepdim=True)) / torch.where(T > 0, T, 1.0))
        best = torch.zeros_like(w).scatter_(1, _first_largest(s), 1.0)
        w = torch.where(T > 0, w, best)
        cum = w.cumsum(-1)
        at = (cum <= st["u"][:, j:j + 1].double() * cum[:, -1:]).sum(-1, keepdim=True).clamp(max=top - 1)
        prev = index[:, j].gather(1, at).squeeze(1)
        chosen.append(prev)
        probs.append(w / w.sum(-1, keepdim=True))
    return torch.stack(chosen, 1).int(), index.int(), torch.stack(probs, 1).float()


def _plain_verify(st):
    c = st["c"]
    b, k, v = c["batch"], c["k"], c["vocab"]
    x, T = st["logits"].double(), st["temperature"].double().view(b, 1, 1)
    greedy = (T <= 0).view(b, 1)
    m, best = x.amax(-1, keepdim=True), _first_largest(x)
    w = torch.exp((x - m) / torch.where(T > 0, T, 1.0))
    p = w / w.sum(-1, keepdim=True)
    n = st["n"].long() if st["n"] is not None else torch.full((b,), k, device="cuda")
    d = st["drafted"].long()
    px = p[:, :k].gather(2, d.unsqueeze(2)).squeeze(2)
    qx = torch.ones_like(px)
    if st["cand"] is not None:
        qx = ((st["cand"] == st["drafted"].unsqueeze(2)) * st["q"].double()).sum(-1)
    good = torch.where(greedy, d == best[:, :k, 0], st["u"][:, :k].double() * qx < px)
    good = good & (torch.arange(k, device="cuda") < n.view(b, 1))
    accepted = good.int().cumprod(1).sum(1)
    p = p.gather(1, accepted.view(b, 1, 1).expand(b, 1, v)).squeeze(1)
    best = best.view(b, k + 1).gather(1, accepted.view(b, 1)).squeeze(1)
    q = torch.zeros_like(p)
    if k:
        at = accepted.clamp(max=k - 1).view(b, 1, 1)
        if st["cand"] is not None:
            cand = st["cand"].long().gather(1, at.expand(b, 1, c["top"])).squeeze(1)
            q.scatter_add_(1, cand, st["q"].double().gather(1, at.expand(b, 1, c["top"])).squeeze(1))
        else:
            q.scatter_(1, d.gather(1, at.view(b, 1)), 1.0)
        q = torch.where((accepted < n).view(b, 1), q, 0.0)
    r = (p - q).clamp(min=0)
    r = torch.where(r.sum(-1, keepdim=True) > 0, r, p)
    cum = r.cumsum(-1)
    token = (cum <= st["u"][:, k:].double() * cum[:, -1:]).sum(-1).clamp(max=v - 1)
    token = torch.where(greedy.view(b), best, token)
    j = torch.arange(k + 1, device="cuda").view(1, -1)
    ids = torch.cat([d, d.new_zeros(b, 1)], 1)
    ids = torch.where(j < accepted.view(b, 1), ids, torch.where(j == accepted.view(b, 1), token.view(b, 1), -1))
    return accepted.int(), ids.int()


# ---------------------------------------------------------------------------------- one pass

def run(state):
    c = state["c"]
    if not own:
        return globals()["_plain_" + c["op"]](state)
    from speculative_block_drafter_gb300 import drafter as D
    if c["op"] == "attend":
        cache = D.KV4Cache.of(state["k"], state["v"], c["hd"])
        return cache.attend(state["q"], state["lo"], state["hi"], state["anchor"], window=c["window"],
                            causal=c["causal"])
    if c["op"] == "write":
        cache = D.KV4Cache.of(state["ck"], state["cv"], c["hd"])
        cache.write(state["at"], state["k"], state["v"])
        return cache.read(state["at"], c["n"])
    if c["op"] == "select":
        return D.select_sample(state["logits"], state["hp"], state["anchor"], state["pred"], state["succ"], c["top"],
                               state["temperature"], state["u"])
    return D.verify(state["logits"], state["drafted"], state["u"], temperature=state["temperature"], cand=state["cand"],
                    cand_q=state["q"], n_drafted=state["n"])


# ---------------------------------------------------------------------------------- the definitions in 64 bits

def _values(buf, row, hd):
    """Rows `row` (a 1-D index) of a cache's bytes [kv][tiles][tile] as f64 [kv][len(row)][hd], value by value."""
    d = torch.arange(hd, device=buf.device)
    t, i = (row // TILE).view(-1, 1), (row % TILE).view(-1, 1)
    e = d % 8
    # nibble e / 2 of the word's low half for an even value, of its high half for an odd one
    byte = (d // 32) * (TILE * 16) + i * 16 + (d % 32) // 8 * 4 + (e % 2) * 2 + e // 4
    code = (buf[:, t, byte].int() >> (4 * (e // 2 % 2))) & 15
    s = TILE * hd // 2 + i * (hd // 16) + (d // 32) * 2
    word = buf[:, t, s].int() | (buf[:, t, s + 1].int() << 8)
    man, ex = (word & 1023).double(), (word >> 10) & 31
    scale = torch.where(ex > 0, torch.ldexp(1 + man / 1024, ex - 15), man * 2.0 ** -24)
    return (code.double() - 8) * scale


def exact(case, seed):
    c = case
    if c["op"] == "verify":
        return None
    st = prepare(case, seed)
    if c["op"] == "attend":
        out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        rep = c["heads"] // c["kv"]
        for b in range(c["batch"]):
            row = torch.arange(st["lo"][b], st["hi"][b], device="cuda")
            k, v = _values(st["k"][b], row, c["hd"]), _values(st["v"][b], row, c["hd"])
            for r in range(c["rows"]):
                pos = st["anchor"][b] + r
                see = torch.ones_like(row, dtype=torch.bool)
                if c["causal"]:
                    see &= row <= pos
                if c["window"]:
                    see &= row > pos - c["window"]
                if not bool(see.any()):
                    continue
                q = st["q"][b, r].double().view(c["kv"], rep, c["hd"])
                s = torch.einsum("ghd,gnd->ghn", q, k) / c["hd"] ** 0.5
                p = torch.softmax(torch.where(see, s, torch.full_like(s, float("-inf"))), -1)
                out[b, r] = torch.einsum("ghn,gnd->ghd", p, v).reshape(c["heads"], c["hd"])
        return out
    if c["op"] == "write":
        out = []
        for x in (st["k"], st["v"]):
            g = x.double().reshape(*x.shape[:-1], c["hd"] // GROUP, GROUP)
            top = g.abs().amax(-1, keepdim=True)
            s = (top / 7).float().bfloat16().half().double()
            # the format rounds the quotient to f32 first
            code = (g / torch.where(s > 0, s, torch.ones_like(s))).float().double().round().clamp(-7, 7)
            out.append((code * s).reshape(x.shape))
        return tuple(out)
    prob = torch.zeros(c["batch"], c["k"], c["top"], dtype=torch.float64)
    # the logits' bits as whole numbers in the values' order, the lower index first among equals
    bits = st["logits"].view(torch.int32).long()
    key = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF)) * (1 << 21) - torch.arange(c["width"], device="cuda")
    cand = key.topk(c["top"], -1).indices
    value, cand = st["logits"].double().gather(2, cand).cpu(), cand.cpu()
    pred, succ, hp = st["pred"].double().cpu(), st["succ"].double().cpu(), st["hp"].double().cpu()
    u, T, prev = st["u"].tolist(), st["temperature"].tolist(), st["anchor"].tolist()
    for b in range(c["batch"]):
        for j in range(c["k"]):
            s = value[b, j] + succ[cand[b, j]] @ (pred[prev[b]] * hp[b, j])
            if T[b] > 0:
                prob[b, j] = torch.softmax(s / T[b], -1)
            else:
                prob[b, j, s.tolist().index(float(s.max()))] = 1
            total, at = 0.0, 0
            for at in range(c["top"]):
                total += float(prob[b, j, at])
                if total > u[b][j]:
                    break
            prev[b] = int(cand[b, j, at])
    return None, None, prob
