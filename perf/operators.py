"""What the cache-compression operators are measured on: a KV cache held in 4 bits
(scatter, read-back, decode attention), decode attention that also accumulates each
token's attention weight, and the eviction of a cache's least attended tokens.

A case is a dict of plain values. prepare() makes what a serving loop has in hand
before the call (queries, a paged cache with shuffled blocks, tables, lengths, output
buffers); run() makes one pass: with `own` false in elementary torch operations, with
`own` true through paged_kv_cache_261_gb300. Lengths are the same set for every seed,
in an order drawn from the seed, so work() needs the case alone.

The 4-bit cache: key_cache, value_cache uint8 [num_blocks, num_kv_heads, block_size,
head_dim / 2] (channel 2i in the low, 2i + 1 in the high half of byte i) and kv_params
float16 [num_blocks, num_kv_heads, block_size, 4] = (K scale, K zero, V scale, V zero)
per token and kv head; a channel stands for code * scale + zero. The 16- and 32-bit
caches: [num_blocks, block_size, num_kv_heads, head_dim].
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BITS = {"bf16": 16, "f16": 16, "f32": 32}


# ---------------------------------------------------------------------------- cases

def listed():
    batch = {"B": 64, "lo": 512, "hi": 4096, "H": 32, "Hk": 8, "D": 128, "bs": 16, "dtype": "bf16", "gain": 1.0}
    long = {"B": 8, "lo": 32768, "hi": 131072, "H": 64, "Hk": 8, "D": 128, "bs": 16, "dtype": "f16", "gain": 2.0}
    return [
        # the write of one decode step of a padded batch: the newest token of 64 sequences, then their read-back
        {"name": "int4_write_step", "kind": "write", "T": 64, "pad": 5, "Hk": 8, "D": 128, "bs": 16, "dtype": "bf16"},
        # a prefill chunk put into the cache and read back for the chunk's own attention
        {"name": "int4_write_chunk", "kind": "write", "T": 8192, "pad": 0, "Hk": 8, "D": 128, "bs": 32,
         "dtype": "f16"},
        # a long cached context expanded to 16 bits ahead of the prefill of its next turn
        {"name": "int4_read_context", "kind": "read", "T": 131071, "pad": 0, "Hk": 8, "D": 128, "bs": 16,
         "dtype": "bf16"},
        # a single interactive request: one short sequence, latency counts
        {"name": "int4_decode_one", "kind": "int4", "B": 1, "lo": 700, "hi": 700, "H": 32, "Hk": 8, "D": 128,
         "bs": 16, "dtype": "bf16", "gain": 1.0, "mass": False},
        # a serving batch of an 8B-shaped model
        dict(batch, name="int4_decode_batch", kind="int4", mass=False),
        # few sequences of very long contexts, eight query heads to a kv head
        dict(long, name="int4_decode_long", kind="int4", mass=False),
        # the serving batch with its attention weights accumulated for a later eviction
        dict(batch, name="int4_decode_scored", kind="int4", mass=True),
        # the same over a 16-bit cache
        dict(batch, name="scored_decode_batch", kind="scored"),
        # the long contexts, where eviction pays most
        dict(long, name="scored_decode_long", kind="scored"),
        # the smallest model that the tests use, in 32 bits
        {"name": "scored_decode_fp32", "kind": "scored", "B": 4, "lo": 5, "hi": 64, "H": 4, "Hk": 4, "D": 64, "bs": 4,
         "dtype": "f32", "gain": 1.0},
        # a serving batch cut back to 1024 tokens a sequence, the newest 128 kept whatever their weight
        dict(batch, name="evict_batch", kind="evict", bits=16, keep=1024, recent=128),
        # long 4-bit contexts cut back to 8192 tokens, then read back for what follows
        dict(long, name="evict_int4_long", kind="evict", bits=4, keep=8192, recent=512, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["write", "read", "int4", "int4", "scored", "scored", "evict", "evict"])
    Hk = rng.choice([1, 2, 4, 8, 8])
    D = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "f16"])
    if kind in ("write", "read"):
        T = _log(rng, 1, 16384 if kind == "write" else 131072)
        return {"kind": kind, "T": T, "pad": rng.randrange(0, 1 + T // 2), "Hk": Hk, "D": D,
                "bs": rng.choice([8, 16, 32, 64]), "dtype": dtype}
    B = _log(rng, 1, 128)
    hi = _log(rng, 24, min(131072, 400000 // B))
    c = {"kind": kind, "B": B, "lo": max(1, hi // rng.choice([1, 3, 9])), "hi": hi, "H": Hk * rng.choice([1, 3, 4, 8]),
         "Hk": Hk, "D": D, "bs": rng.choice([8, 16, 32, 64]), "dtype": dtype, "gain": rng.choice([1.0, 2.0])}
    if kind == "int4":
        c["mass"] = rng.random() < 0.5
    elif kind == "scored":
        c["dtype"] = rng.choice(["bf16", "f16", "f32"])
    else:
        c["bits"] = rng.choice([4, 16])
        c["keep"] = _log(rng, 8, min(hi, 8192))
        c["recent"] = rng.randrange(0, c["keep"] + 1)
    return c


def _lengths(case):
    """The context lengths of a case, spread over [lo, hi], both ends among them; the same for every seed."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi] + [lo + int((hi - lo) * ((b * 0.6180339887498949) % 1.0)) for b in range(B - 1)]


def _kept(case):
    return [min(n, case["keep"]) for n in _lengths(case)]


def _blocks(n, bs):
    return -(-n // bs)


def work(case):
    """Each input read once, each output written once; a cache counts where its tokens lie in a context."""
    kind, Hk, D = case["kind"], case["Hk"], case["D"]
    es = _BITS[case["dtype"]] // 8
    row4 = 2 * (D // 2) + 8                           # a token's codes and parameters of one kv head, K and V
    if kind in ("write", "read"):
        T = case["T"] - case["pad"]
        rows = T * Hk
        wide = 2 * rows * D * es
        if kind == "read":
            return {"bytes": wide + rows * row4 + 4 * case["T"], "flops": 4 * rows * D}
        # the chunk in, its codes written and read back, the values out
        return {"bytes": 2 * wide + 2 * rows * row4 + 4 * case["T"], "flops": 12 * rows * D}
    lens = _lengths(case)
    total = sum(lens)
    tables = 4 * sum(_blocks(n, case["bs"]) for n in lens) + 4 * len(lens)
    if kind == "evict":
        kept = _kept(case)
        moved = sum(kept) * Hk
        row = row4 if case["bits"] == 4 else 2 * D * es
        n = total * Hk * 4 + 2 * moved * row + moved * 8 + tables + 4 * sum(_blocks(n, case["bs"]) for n in kept)
        if case["bits"] == 4:
            n += moved * (row4 + 2 * D * es)          # the read-back
        return {"bytes": n, "flops": total * Hk}
    row = row4 if kind == "int4" else 2 * D * es
    n = total * Hk * row + 2 * case["B"] * case["H"] * D * es + tables
    if kind == "scored" or case.get("mass"):
        n += total * Hk * 8                           # the accumulated weights, read and written
    return {"bytes": n, "flops": 4 * total * case["H"] * D}


# ---------------------------------------------------------------------------- inputs

def _quantise(x):
    """Codes (uint8, unpacked), scales and zeros (float16) of rows x [..., D], in float32 throughout."""
    x = x.float().clamp(-65504.0, 65504.0)
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    zero = lo.half()
    scale = ((hi - lo) / 15.0).half()
    s = scale.float()
    n = torch.round((x - zero.float()) / torch.where(s > 0, s, torch.ones_like(s))).clamp(0.0, 15.0)
    return torch.where(s > 0, n, torch.zeros_like(n)).to(torch.uint8), scale.squeeze(-1), zero.squeeze(-1)


def _pack(n):
    return n[..., 0::2] | (n[..., 1::2] << 4)


def _unpack(b):
    return torch.stack((b & 15, b >> 4), -1).flatten(-2)


def _rows(g, shape, dev, which):
    """Rows like a projection's output: channels of unequal size and, for K, of unequal mean."""
    D = shape[-1]
    size = 0.5 + torch.rand(D, generator=g, device=dev)
    x = torch.randn(shape, generator=g, device=dev) * size
    return x + 0.5 * torch.randn(D, generator=g, device=dev) if which == "k" else x


def _cache4(g, nb, Hk, bs, D, dev):
    kc = torch.empty((nb, Hk, bs, D // 2), dtype=torch.uint8, device=dev)
    vc = torch.empty_like(kc)
    par = torch.empty((nb, Hk, bs, 4), dtype=torch.float16, device=dev)
    step = max(1, (1 << 26) // (Hk * bs * D))
    for a in range(0, nb, step):
        e = min(nb, a + step)
        for j, (c, which) in enumerate(((kc, "k"), (vc, "v"))):
            n, s, z = _quantise(_rows(g, (e - a, Hk, bs, D), dev, which))
            c[a:e] = _pack(n)
            par[a:e, :, :, 2 * j] = s
            par[a:e, :, :, 2 * j + 1] = z
    return kc, vc, par


def _cache(g, nb, Hk, bs, D, dtype, dev):
    kc = torch.empty((nb, bs, Hk, D), dtype=dtype, device=dev)
    vc = torch.empty_like(kc)
    step = max(1, (1 << 26) // (Hk * bs * D))
    for a in range(0, nb, step):
        e = min(nb, a + step)
        kc[a:e] = _rows(g, (e - a, bs, Hk, D), dev, "k").to(dtype)
        vc[a:e] = _rows(g, (e - a, bs, Hk, D), dev, "v").to(dtype)
    return kc, vc


def _table(perm, first, lens, bs, dev):
    """Block table [B, MB] of `lens` tokens a row taken from perm[first:], padded with -1; and the blocks taken."""
    need = torch.tensor([_blocks(n, bs) for n in lens], device=dev)
    width = max(1, int(need.max()))
    start = torch.cumsum(need, 0) - need
    j = torch.arange(width, device=dev)
    at = (first + start[:, None] + j).clamp(max=perm.numel() - 1)
    used = int(need.sum())
    return torch.where(j < need[:, None], perm[at], torch.full_like(at, -1)).to(torch.int32), used


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    Hk, D, bs, dtype = case["Hk"], case["D"], case["bs"], _DTYPES[case["dtype"]]
    s = {"case": case}
    if case["kind"] in ("write", "read"):
        T = case["T"]
        nb = _blocks(T, bs) + 1 + _blocks(T, 8 * bs)
        slots = torch.randperm(nb * bs, generator=g, device=dev)[:T].to(torch.int32)
        if case["kind"] == "read":               # a context: whole blocks in shuffled order
            perm = torch.randperm(nb, generator=g, device=dev)
            t = torch.arange(T, device=dev)
            slots = (perm[t // bs] * bs + t % bs).to(torch.int32)
        if case["pad"]:
            slots[T - case["pad"]:] = -1
        s["slots"] = slots
        s["kc"], s["vc"], s["par"] = _cache4(g, nb, Hk, bs, D, dev)
        if case["kind"] == "write":
            s["k"] = _rows(g, (T, Hk, D), dev, "k").to(dtype)
            s["v"] = _rows(g, (T, Hk, D), dev, "v").to(dtype)
        s["k_out"] = torch.zeros((T, Hk, D), dtype=dtype, device=dev)
        s["v_out"] = torch.zeros_like(s["k_out"])
        return s
    B, H = case["B"], case["H"]
    order = torch.randperm(B, generator=g, device=dev).tolist()
    base = _lengths(case)
    lens = [base[i] for i in order]
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["max_len"] = max(lens)
    kept = [min(n, case.get("keep", 0)) for n in lens]
    need = sum(_blocks(n, bs) for n in lens) + sum(_blocks(n, bs) for n in kept)
    nb = need + need // 10 + 1
    perm = torch.randperm(nb, generator=g, device=dev)
    s["table"], used = _table(perm, 0, lens, bs, dev)
    if case["kind"] == "int4" or case.get("bits") == 4:
        s["kc"], s["vc"], s["par"] = _cache4(g, nb, Hk, bs, D, dev)
    else:
        s["kc"], s["vc"] = _cache(g, nb, Hk, bs, D, dtype, dev)
    if case["kind"] == "scored" or case.get("mass") or case["kind"] == "evict":
        # weights accumulated over earlier steps: a few tokens hold most of them; zero past each context
        m = torch.rand((B, Hk, max(lens)), generator=g, device=dev)
        m = 0.01 * m + torch.rand(m.shape, generator=g, device=dev).pow(24)
        s["mass"] = m * (torch.arange(max(lens), device=dev) < s["lens"][:, None, None])
    if case["kind"] == "evict":
        s["keep"] = torch.tensor([case["keep"]] * B, dtype=torch.int32, device=dev)
        s["out_table"], _ = _table(perm, used, kept, bs, dev)
        s["kept"] = torch.empty((B, Hk, max(kept)), dtype=torch.int32, device=dev)
        s["mass_out"] = torch.zeros((B, Hk, max(kept)), device=dev)
        if case["bits"] == 4:
            t = torch.arange(max(kept), device=dev)
            slots = s["out_table"].long()[:, t // bs] * bs + t % bs
            live = t < torch.tensor(kept, device=dev)[:, None]
            s["slots"] = torch.where(live, slots, torch.full_like(slots, -1)).flatten().to(torch.int32)
            s["k_out"] = torch.zeros((B * max(kept), Hk, D), dtype=dtype, device=dev)
            s["v_out"] = torch.zeros_like(s["k_out"])
        return s
    s["scale"] = D ** -0.5
    s["q"] = (torch.randn((B, H, D), generator=g, device=dev) * case["gain"]).to(dtype)
    s["out"] = torch.empty_like(s["q"])
    return s


# ---------------------------------------------------------------------------- one pass

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import paged_kv_cache_261_gb300 as pa
    case = s["case"]
    kind = case["kind"]
    if kind in ("write", "read"):
        if kind == "write":
            pa.paged_kv_write_int4(s["k"], s["v"], s["slots"], s["kc"], s["vc"], s["par"])
        pa.paged_kv_read_int4(s["k_out"], s["v_out"], s["slots"], s["kc"], s["vc"], s["par"])
        return s["k_out"], s["v_out"]
    if kind == "int4":
        pa.paged_attention_decode_int4(s["out"], s["q"], s["kc"], s["vc"], s["par"], s["table"], s["lens"], s["scale"],
                                       max_context_len=s["max_len"], mass=s.get("mass"))
        return (s["out"], s["mass"]) if case["mass"] else s["out"]
    if kind == "scored":
        pa.paged_attention_decode_scored(s["out"], s["q"], s["mass"], s["kc"], s["vc"], s["table"], s["lens"],
                                         s["scale"], max_context_len=s["max_len"])
        return s["out"], s["mass"]
    pa.paged_kv_evict(s["kept"], s["mass"], s["mass_out"], s["kc"], s["vc"], s["table"], s["out_table"], s["lens"],
                      s["keep"], case["recent"], kv_params=s.get("par"))
    if case["bits"] == 4:
        pa.paged_kv_read_int4(s["k_out"], s["v_out"], s["slots"], s["kc"], s["vc"], s["par"])
        return s["kept"], s["mass_out"], s["k_out"], s["v_out"]
    return s["kept"], s["mass_out"], s["kc"], s["vc"]


def _read4(s, slots):
    """K and V values in float32 of the 4-bit cache at `slots` [n]: two [n, Hk, D]."""
    bs = s["case"]["bs"]
    block, off = slots // bs, slots % bs
    par = s["par"][block, :, off].float()
    k = _unpack(s["kc"][block, :, off]).float() * par[..., 0:1] + par[..., 1:2]
    v = _unpack(s["vc"][block, :, off]).float() * par[..., 2:3] + par[..., 3:4]
    return k, v


def _slots_of(table, n, bs):
    """Slot of each of the first n positions of every sequence, [B, n]; padded entries read as block 0."""
    t = torch.arange(n, device=table.device)
    return table.long().clamp(min=0)[:, t // bs] * bs + t % bs


def _plain(s):
    case = s["case"]
    kind, bs = case["kind"], case["bs"]
    if kind in ("write", "read"):
        live = s["slots"] >= 0
        slots = s["slots"].long()[live]
        if kind == "write":
            block, off = slots // bs, slots % bs
            nk, sk, zk = _quantise(s["k"][live])
            nv, sv, zv = _quantise(s["v"][live])
            s["kc"][block, :, off] = _pack(nk)
            s["vc"][block, :, off] = _pack(nv)
            s["par"][block, :, off] = torch.stack((sk, zk, sv, zv), -1)
        k, v = _read4(s, slots)
        s["k_out"][live] = k.to(s["k_out"].dtype)
        s["v_out"][live] = v.to(s["v_out"].dtype)
        return s["k_out"], s["v_out"]
    if kind == "evict":
        return _plain_evict(s)
    B, H, D = s["q"].shape
    Hk, n = case["Hk"], s["max_len"]
    slots = _slots_of(s["table"], n, bs)
    if kind == "int4":
        k, v = _read4(s, slots.flatten())
    else:
        k = s["kc"].flatten(0, 1)[slots.flatten()].float()
        v = s["vc"].flatten(0, 1)[slots.flatten()].float()
    k = k.view(B, n, Hk, D).permute(0, 2, 3, 1)                       # [B, Hk, D, n]
    v = v.view(B, n, Hk, D).permute(0, 2, 1, 3)                       # [B, Hk, n, D]
    q = s["q"].float().view(B, Hk, H // Hk, D)
    x = torch.matmul(q, k) * s["scale"]
    x = x.masked_fill(torch.arange(n, device=x.device) >= s["lens"][:, None, None, None], -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    w = e / e.sum(-1, keepdim=True)
    out = torch.matmul(w, v).reshape(B, H, D).to(s["q"].dtype)
    if kind == "scored" or case["mass"]:
        s["mass"] += w.sum(2)
        return out, s["mass"]
    return out


def _plain_evict(s):
    case = s["case"]
    bs, mass, Hk = case["bs"], s["mass"], case["Hk"]
    B, n = mass.shape[0], mass.shape[2]
    t = torch.arange(n, device=mass.device)
    c = s["lens"].long()[:, None, None]
    keep = torch.minimum(s["keep"].long()[:, None, None], c)          # tokens that stay
    recent = torch.minimum(torch.full_like(keep, case["recent"]), keep)
    old = t < c - recent                                               # those that compete
    order = torch.sort(mass.masked_fill(~old, -math.inf), dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, t.expand_as(order).contiguous())
    stays = (old & (rank < keep - recent)) | ((t >= c - recent) & (t < c))
    m = s["kept"].shape[2]
    to = torch.where(stays, stays.cumsum(-1) - 1, torch.full_like(order, m))
    kept = torch.full((B, Hk, m + 1), -1, dtype=torch.long, device=mass.device)
    kept.scatter_(-1, to, t.expand_as(to).contiguous())
    kept = kept[..., :m]
    live = kept >= 0
    src = kept.clamp(min=0)
    s["kept"].copy_(kept)
    s["mass_out"].copy_(torch.where(live, mass.gather(-1, src), torch.zeros_like(s["mass_out"])))
    row = torch.arange(B, device=mass.device)[:, None, None]
    j = torch.arange(m, device=mass.device)
    head = torch.arange(Hk, device=mass.device)[None, :, None].expand_as(src)[live]
    sb = s["table"].long()[row, src // bs][live]
    so = (src % bs)[live]
    db = s["out_table"].long()[row, (j // bs).expand_as(src)][live]
    do = (j % bs).expand_as(src)[live]
    if case["bits"] == 4:
        s["kc"][db, head, do] = s["kc"][sb, head, so]
        s["vc"][db, head, do] = s["vc"][sb, head, so]
        s["par"][db, head, do] = s["par"][sb, head, so]
        ok = s["slots"] >= 0
        k, v = _read4(s, s["slots"].long()[ok])
        s["k_out"][ok] = k.to(s["k_out"].dtype)
        s["v_out"][ok] = v.to(s["v_out"].dtype)
        return s["kept"], s["mass_out"], s["k_out"], s["v_out"]
    s["kc"][db, do, head] = s["kc"][sb, so, head]
    s["vc"][db, do, head] = s["vc"][sb, so, head]
    return s["kept"], s["mass_out"], s["kc"], s["vc"]


# ---------------------------------------------------------------------------- in 64 bits

def _codes64(x):
    """The 4-bit format's values of rows x, in 64 bits: the codes follow from float32 differences and quotients."""
    x = x.double().clamp(-65504.0, 65504.0)
    low, high = x.min(-1).values, x.max(-1).values
    zero = low.float().half().double()
    scale = ((high - low).float().double() / 15.0).float().half().double()
    d = (x - zero[..., None]).float().double()
    safe = torch.where(scale > 0, scale, torch.ones_like(scale))[..., None]
    n = torch.round((d / safe).float().double()).clamp(0.0, 15.0) * (scale > 0)[..., None]
    return n * scale[..., None] + zero[..., None]


def _value64(codes, par, which):
    byte = codes.long()
    n = torch.empty((*byte.shape[:-1], 2 * byte.shape[-1]), dtype=torch.float64, device=byte.device)
    n[..., 0::2] = (byte % 16).double()
    n[..., 1::2] = (byte // 16).double()
    p = par.double()
    return n * p[..., 2 * which, None] + p[..., 2 * which + 1, None]


def exact(case, seed):
    s = prepare(case, seed)
    kind, bs = case["kind"], case["bs"]
    if kind in ("write", "read"):
        out = [s["k_out"].double(), s["v_out"].double()]
        for a in range(0, case["T"] - case["pad"], 16384):
            e = min(case["T"] - case["pad"], a + 16384)
            slot = s["slots"][a:e].long()
            b, o = torch.div(slot, bs, rounding_mode="floor"), slot.remainder(bs)
            for i, (new, cache) in enumerate((("k", "kc"), ("v", "vc"))):
                out[i][a:e] = (_codes64(s[new][a:e]) if kind == "write"
                               else _value64(s[cache][b, :, o], s["par"][b, :, o], i))
        return tuple(out)
    if kind == "evict":
        return _exact_evict(s)
    B, H, D = s["q"].shape
    Hk = case["Hk"]
    G = H // Hk
    out = torch.zeros((B, H, D), dtype=torch.float64, device=s["q"].device)
    mass = s["mass"].double() if "mass" in s else None
    for b in range(B):
        n = int(s["lens"][b])
        blk = s["table"][b, :_blocks(n, bs)].long()
        for h in range(Hk):
            if kind == "int4":
                k = _value64(s["kc"][blk, h], s["par"][blk, h], 0).reshape(-1, D)[:n]
                v = _value64(s["vc"][blk, h], s["par"][blk, h], 1).reshape(-1, D)[:n]
            else:
                k = s["kc"][blk, :, h].reshape(-1, D)[:n].double()
                v = s["vc"][blk, :, h].reshape(-1, D)[:n].double()
            w = torch.softmax(k @ s["q"][b, h * G:(h + 1) * G].double().t() * s["scale"], 0)   # [n, G]
            out[b, h * G:(h + 1) * G] = w.t() @ v
            if mass is not None:
                mass[b, h, :n] += w.sum(1)
    return (out, mass) if mass is not None else out


def _exact_evict(s):
    case = s["case"]
    bs, Hk = case["bs"], case["Hk"]
    mass = s["mass"].cpu().double().numpy()
    mass_out = torch.zeros(s["mass_out"].shape, dtype=torch.float64)
    four = case["bits"] == 4
    if four:
        k, v = (torch.zeros(s[x].shape, dtype=torch.float64, device=s[x].device) for x in ("k_out", "v_out"))
    else:
        k, v = s["kc"].double(), s["vc"].double()
    m = s["kept"].shape[2]
    for b, c in enumerate(s["lens"].tolist()):
        n = min(c, case["keep"])
        r = min(case["recent"], n)
        for h in range(Hk):
            first = (-mass[b, h, :c - r]).argsort(kind="stable")[:n - r]     # heaviest first, ties to the lower index
            at = torch.tensor(sorted(first.tolist()) + list(range(c - r, c)), dtype=torch.long)
            mass_out[b, h, :n] = torch.from_numpy(mass[b, h][at.numpy()])
            at = at.to(s["table"].device)
            j = torch.arange(n, device=at.device)
            sb, db = s["table"][b, at // bs].long(), s["out_table"][b, j // bs].long()
            if four:
                par = s["par"][sb, h, at % bs]
                k[b * m:b * m + n, h] = _value64(s["kc"][sb, h, at % bs], par, 0)
                v[b * m:b * m + n, h] = _value64(s["vc"][sb, h, at % bs], par, 1)
            else:
                k[db, j % bs, h] = s["kc"][sb, at % bs, h].double()
                v[db, j % bs, h] = s["vc"][sb, at % bs, h].double()
    return None, mass_out.to(s["mass"].device), k, v
