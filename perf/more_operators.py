"""What the operators of a serving step over a block-scaled 8-bit cache are measured on:
block tables and slot maps built on the GPU from the requests' lengths, rotary positions
(with the scatter of the rotated keys), the scatter and read-back of an 8-bit cache that
has a scale for each block of tokens and kv head, and decode attention over it.

A case is a dict of plain values. prepare() makes what a serving loop has in hand before
the call (projections, a paged cache with shuffled blocks, tables, lengths, output buffers);
run() makes one pass: with `own` false in elementary torch operations, with `own` true
through paged_kv_cache_261_gb300. Lengths are the same set for every seed, in an order drawn
from the seed, so work() needs the case alone.

The block-scaled cache: key_cache, value_cache uint8 [num_blocks, num_kv_heads, block_size,
head_dim] of E4M3 codes and kv_scales float32 [num_blocks, num_kv_heads, 2] = (K scale, V
scale); a channel stands for code * scale. Writing a token makes a block's scale the smallest
power of two 2^e, e >= -100, for which the block's largest finite magnitude is at most 448 * 2^e;
when that grows, the codes that the block held before are re-encoded, and a call that writes a block's first slot
starts the block anew. The caches of the rotary cases: [num_blocks, block_size, num_kv_heads,
head_dim] in 16 or 32 bits.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ---------------------------------------------------------------------------- cases

def listed():
    heads = {"H": 32, "Hk": 8, "D": 128, "bs": 16}
    return [
        # the metadata of one decode step: 64 requests with a token each, four others just finished
        {"name": "layout_step", "kind": "layout", "B": 64, "lo": 512, "hi": 4096, "chunk": 1, "chunks": 0, "done": 4,
         "bs": 16, "short": False},
        # a mixed step: a third of 192 requests has a prefill chunk of up to 512 tokens, the others a token each
        {"name": "layout_mixed", "kind": "layout", "B": 192, "lo": 0, "hi": 8192, "chunk": 512, "chunks": 64, "done": 5,
         "bs": 16, "short": False},
        # the largest: 1024 requests, half of them with a prefill chunk, and a pool that runs dry on the way
        {"name": "layout_large", "kind": "layout", "B": 1024, "lo": 0, "hi": 16384, "chunk": 512, "chunks": 512,
         "done": 30, "bs": 32, "short": True},
        # the queries and keys of one decode step of a padded batch, rotated, and the keys and values stored
        dict(heads, name="rotary_step", kind="rotary", T=64, pad=5, dtype="bf16", rd=128, pairs="half",
             scaling="none", far=4096, store=True),
        # a prefill chunk; interleaved pairs in the first half of every head
        dict(heads, name="rotary_chunk", kind="rotary", T=8192, pad=0, dtype="f16", rd=64, pairs="interleaved",
             scaling="ntk", far=32768, store=True),
        # a chunk far out in a long context, frequencies scaled for it; its keys go on to a cache of fewer bits
        dict(heads, H=64, name="rotary_far", kind="rotary", T=2047, pad=0, dtype="bf16", rd=128, pairs="half",
             scaling="by_turns", far=1048576, store=False),
        # the newest token of 64 sequences written into their last blocks, those blocks read back
        {"name": "blk8_write_step", "kind": "write", "B": 64, "lo": 512, "hi": 4096, "new": 1, "pad": 5, "Hk": 8,
         "D": 128, "bs": 16, "dtype": "bf16"},
        # prefill chunks of four prompts written and read back for the chunks' own attention
        {"name": "blk8_write_chunk", "kind": "write", "B": 4, "lo": 0, "hi": 6000, "new": 2048, "pad": 0, "Hk": 8,
         "D": 128, "bs": 32, "dtype": "f16"},
        # a long cached context expanded to 16 bits ahead of the prefill of its next turn
        {"name": "blk8_read_context", "kind": "read", "T": 131071, "Hk": 8, "D": 128, "bs": 16, "dtype": "bf16"},
        # a single interactive request: one short sequence, latency counts
        dict(heads, name="blk8_decode_one", kind="decode", B=1, lo=700, hi=700, dtype="bf16", gain=1.0),
        # a serving batch of an 8B-shaped model
        dict(heads, name="blk8_decode_batch", kind="decode", B=64, lo=512, hi=4096, dtype="bf16", gain=1.0),
        # few sequences of very long contexts, eight query heads to a kv head
        dict(heads, H=64, name="blk8_decode_long", kind="decode", B=8, lo=32768, hi=131072, dtype="f16", gain=2.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["layout", "rotary", "rotary", "write", "read", "decode", "decode", "decode"])
    bs = rng.choice([8, 16, 32, 64])
    Hk = rng.choice([1, 2, 4, 8, 8])
    D = rng.choice([64, 128, 128])
    if kind == "layout":
        B = _log(rng, 1, 1024)
        hi = _log(rng, 1, 16384)
        return {"kind": kind, "B": B, "lo": rng.randrange(0, hi + 1), "hi": hi, "chunk": _log(rng, 1, 512),
                "chunks": rng.randrange(0, B // 2 + 1), "done": rng.randrange(0, B // 4 + 1), "bs": bs,
                "short": rng.random() < 0.3}
    if kind == "rotary":
        T = _log(rng, 1, 8192)
        return {"kind": kind, "T": T, "pad": rng.randrange(0, 1 + T // 2), "H": Hk * rng.choice([1, 3, 4]), "Hk": Hk,
                "D": D, "bs": bs, "dtype": rng.choice(["bf16", "f16", "f32"]), "rd": rng.choice([16, 32, 48, 64, D]),
                "pairs": rng.choice(["half", "interleaved"]),
                "scaling": rng.choice(["none", "linear", "ntk", "by_turns", "by_index"]), "far": _log(rng, 16, 1048576),
                "store": rng.random() < 0.7}
    if kind == "read":
        return {"kind": kind, "T": _log(rng, 1, 131072), "Hk": Hk, "D": D, "bs": bs, "dtype": rng.choice(["bf16", "f16", "f32"])}
    if kind == "write":
        B = _log(rng, 1, 128)
        hi = _log(rng, 1, 4096)
        new = _log(rng, 1, 8192 // B)
        return {"kind": kind, "B": B, "lo": rng.randrange(0, hi + 1), "hi": hi, "new": new, "pad": rng.randrange(0, 6),
                "Hk": Hk, "D": D, "bs": bs, "dtype": rng.choice(["bf16", "f16", "f32"])}
    B = _log(rng, 1, 128)
    hi = _log(rng, 24, min(131072, 400000 // B))
    return {"kind": kind, "B": B, "lo": rng.choice([0, hi, hi // 3, hi // 9]), "hi": hi,
            "H": Hk * rng.choice([1, 3, 4, 8, 16]), "Hk": Hk, "D": D, "bs": bs, "dtype": rng.choice(["bf16", "f16"]),
            "gain": rng.choice([1.0, 2.0])}


def _spread(n, lo, hi):
    """n lengths over [lo, hi], both ends among them; the same for every seed."""
    return [hi] + [lo + int((hi - lo) * ((b * 0.6180339887498949) % 1.0)) for b in range(n - 1)]


def _lengths(case):
    return _spread(case["B"], case["lo"], case["hi"])


def _new_tokens(case):
    """New tokens of each request of a layout case: none for the finished, then chunks, then single tokens."""
    chunks = _spread(case["chunks"], 1, case["chunk"]) if case["chunks"] else []
    return [0] * case["done"] + chunks + [1] * (case["B"] - case["done"] - case["chunks"])


def _blocks(n, bs):
    return -(-n // bs)


def _touched(case):
    """Tokens of a write case in the blocks that it writes to, a sequence each."""
    bs, new = case["bs"], case["new"]
    return [c % bs + new for c in _lengths(case)]


def work(case):
    """Each input read once, each output written once; a cache counts where its tokens lie in a context."""
    kind, bs = case["kind"], case["bs"]
    if kind == "layout":
        B, lens, new = case["B"], _lengths(case), _new_tokens(case)
        T = sum(new)
        moved = sum(_blocks(n, bs) for n in lens[:case["done"]]) + sum(_blocks(n, bs) for n in new)
        # lengths, new lengths and starts; slots and positions; blocks given back and taken
        return {"bytes": 25 * B + 8 * T + 12 * moved, "flops": 10 * (T + B)}
    Hk, D, es = case["Hk"], case["D"], _BYTES[case["dtype"]]
    if kind == "rotary":
        T, H, rd = case["T"], case["H"], case["rd"]
        rows = T * (H + Hk)
        stored = T - case["pad"] if case["store"] else 0
        n = 2 * rows * D * es + 2 * stored * Hk * D * es + 8 * T + 4 * rd
        return {"bytes": n - (0 if not case["store"] else case["pad"] * Hk * D * es), "flops": 3 * rows * rd + 20 * T * rd}
    if kind in ("write", "read"):
        if kind == "read":
            T = case["T"]
            return {"bytes": T * Hk * 2 * D * (1 + es) + 4 * T + _blocks(T, bs) * Hk * 8, "flops": 2 * T * Hk * D}
        T, near = case["B"] * case["new"], sum(_touched(case))
        blocks = sum(_blocks(n, bs) for n in _touched(case))
        # the new tokens in and encoded, their blocks' tokens read back
        n = T * Hk * 2 * D * (es + 1) + near * Hk * 2 * D * (1 + es) + 4 * (T + near) + blocks * Hk * 24
        return {"bytes": n, "flops": 4 * T * Hk * D + 2 * near * Hk * D}
    lens, H = _lengths(case), case["H"]
    blocks = sum(_blocks(n, bs) for n in lens)
    n = sum(lens) * Hk * 2 * D + blocks * (Hk * 8 + 4) + 4 * len(lens) + 2 * case["B"] * H * D * es
    return {"bytes": n, "flops": 4 * sum(lens) * H * D}


# ---------------------------------------------------------------------------- inputs

def _rows(g, shape, dev, which):
    """Rows like a projection's output: channels of unequal size and, for K, of unequal mean."""
    D = shape[-1]
    size = 0.5 + torch.rand(D, generator=g, device=dev)
    x = torch.randn(shape, generator=g, device=dev) * size
    return x + 0.5 * torch.randn(D, generator=g, device=dev) if which == "k" else x


def _scale_for(amax):
    """The smallest 2^e, e >= -100, with amax <= 448 * 2^e, in float32."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, -100)).clamp(min=-100)
    return ((e.int() + 127) << 23).view(torch.float32)


def _codes(x):
    """E4M3 codes (uint8) of float32 x, |x| <= 448."""
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def _values(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _cache8(g, nb, Hk, bs, D, dev):
    """Blocks of unequal size, encoded block by block."""
    kc = torch.empty((nb, Hk, bs, D), dtype=torch.uint8, device=dev)
    vc = torch.empty_like(kc)
    scales = torch.empty((nb, Hk, 2), dtype=torch.float32, device=dev)
    step = max(1, (1 << 26) // (Hk * bs * D))
    for a in range(0, nb, step):
        e = min(nb, a + step)
        for j, (c, which) in enumerate(((kc, "k"), (vc, "v"))):
            x = _rows(g, (e - a, Hk, bs, D), dev, which)
            x *= torch.exp2(torch.rand((e - a, Hk, 1, 1), generator=g, device=dev) * 2 - 1)
            s = _scale_for(x.abs().amax((2, 3)))
            c[a:e] = _codes(x / s[:, :, None, None])
            scales[a:e, :, j] = s
    return kc, vc, scales


def _table(perm, lens, width, bs, dev):
    """Block table [B, width] of `lens` tokens a row taken from perm, padded with -1; and the blocks taken."""
    need = torch.tensor([_blocks(n, bs) for n in lens], device=dev)
    start = torch.cumsum(need, 0) - need
    j = torch.arange(width, device=dev)
    at = (start[:, None] + j).clamp(max=perm.numel() - 1)
    return torch.where(j < need[:, None], perm[at], torch.full_like(at, -1)).to(torch.int32), int(need.sum())


def _slots_at(table, row, pos, bs):
    return (table[row, pos // bs].long() * bs + pos % bs).to(torch.int32)


def _frequencies(case):
    """Radians per position of every pair, as a model's configuration gives them: plain, or scaled by 8 for
    contexts beyond 8192 tokens."""
    rd, base, factor, L = case["rd"], 10000.0, 8.0, 8192
    kind = case["scaling"]
    if kind == "ntk" and rd > 2:
        base *= factor ** (rd / (rd - 2))
    f = [base ** (-2.0 * j / rd) for j in range(rd // 2)]
    if kind == "linear":
        f = [x / factor for x in f]
    if kind == "by_turns":                       # slow pairs stretched, fast ones kept, by their turns over L tokens
        keep = [min(1.0, max(0.0, (L * x / (2 * math.pi) - 1.0) / (4.0 - 1.0))) for x in f]
        f = [x / factor * (1 - k) + x * k for x, k in zip(f, keep)]
    if kind == "by_index":                       # the same with a ramp over the pairs' indices
        at = [rd * math.log(L / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rd // 2 - 1)
        keep = [1.0 - min(1.0, max(0.0, (j - lo) / max(hi - lo, 0.001))) for j in range(rd // 2)]
        f = [x / factor * (1 - k) + x * k for x, k in zip(f, keep)]
    return f, (0.1 * math.log(factor) + 1.0 if kind == "by_index" else 1.0)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    bs, s = case["bs"], {"case": case}
    make = {"layout": _prepare_layout, "rotary": _prepare_rotary, "write": _prepare_write, "read": _prepare_read,
            "decode": _prepare_decode}[case["kind"]]
    make(case, s, g, dev, bs)
    return s


def _i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _prepare_layout(case, s, g, dev, bs):
    B, lens, new = case["B"], _lengths(case), _new_tokens(case)
    order = torch.randperm(B, generator=g, device=dev).tolist()
    lens, new, done = [lens[i] for i in order], [new[i] for i in order], [i < case["done"] for i in order]
    held = sum(_blocks(n, bs) for n in lens)
    back = sum(_blocks(n, bs) for n, d in zip(lens, done) if d)
    want = sum(_blocks(c + n, bs) - _blocks(c, bs) for c, n in zip(lens, new))
    free = max(0, want * 2 // 3 - back) if case["short"] else want + want // 4 + 8
    nb = held + free
    perm = torch.randperm(max(nb, 1), generator=g, device=dev)
    width = max(1, max(_blocks(c + n, bs) for c, n in zip(lens, new)))
    s["table"], used = _table(perm, lens, width, bs, dev)
    s["nb"] = max(nb, 1)
    s["lens"], s["new"], s["done"] = _i32(lens, dev), _i32(new, dev), torch.tensor(done, device=dev)
    s["free"] = torch.full((s["nb"],), -1, dtype=torch.int32, device=dev)
    s["free"][:free] = perm[used:used + free].to(torch.int32)
    s["num_free"] = _i32([free], dev)
    s["lens_1"], s["lens_2"] = torch.zeros_like(s["lens"]), torch.zeros_like(s["lens"])
    s["num_free_1"], s["num_free_2"] = torch.zeros_like(s["num_free"]), torch.zeros_like(s["num_free"])
    T = sum(new)
    s["start"] = torch.zeros(B + 1, dtype=torch.int32, device=dev)
    s["slots"] = torch.zeros(max(1, T + T // 16), dtype=torch.int32, device=dev)      # padded, as a captured step's
    s["positions"] = torch.zeros_like(s["slots"])


def _prepare_rotary(case, s, g, dev, bs):
    T, H, Hk, D, dtype = case["T"], case["H"], case["Hk"], case["D"], _DTYPES[case["dtype"]]
    # one fused projection: q, k and v are views of its rows
    x = _rows(g, (T, H + 2 * Hk, D), dev, "k").to(dtype)
    s["q"], s["k"], s["v"] = x[:, :H], x[:, H:H + Hk], x[:, H + Hk:]
    s["positions"] = torch.randint(0, case["far"], (T,), generator=g, device=dev, dtype=torch.int32)
    f, s["factor"] = _frequencies(case)
    s["inv_freq"] = torch.tensor(f, dtype=torch.float64, device=dev)
    s["q_out"] = torch.empty((T, H, D), dtype=dtype, device=dev)
    if not case["store"]:
        s["k_out"] = torch.empty((T, Hk, D), dtype=dtype, device=dev)
        return
    nb = _blocks(T, bs) + 1 + _blocks(T, 8 * bs)
    s["slots"] = torch.randperm(nb * bs, generator=g, device=dev)[:T].to(torch.int32)
    if case["pad"]:
        s["slots"][T - case["pad"]:] = -1
    s["kc"] = torch.zeros((nb, bs, Hk, D), dtype=dtype, device=dev)
    s["vc"] = torch.zeros_like(s["kc"])


def _prepare_write(case, s, g, dev, bs):
    B, Hk, D, dtype, new = case["B"], case["Hk"], case["D"], _DTYPES[case["dtype"]], case["new"]
    base = _lengths(case)
    lens = [base[i] for i in torch.randperm(B, generator=g, device=dev).tolist()]
    nb = sum(_blocks(n + new, bs) for n in lens) + 2
    perm = torch.randperm(nb, generator=g, device=dev)
    table, _ = _table(perm, [n + new for n in lens], max(_blocks(n + new, bs) for n in lens), bs, dev)
    c = torch.tensor(lens, device=dev)
    row = torch.arange(B, device=dev)[:, None]
    slots = _slots_at(table, row, c[:, None] + torch.arange(new, device=dev), bs).flatten()
    s["slots"] = torch.cat((slots, torch.full((case["pad"],), -1, dtype=torch.int32, device=dev)))
    T = s["slots"].numel()
    s["kc"], s["vc"], s["scales"] = _cache8(g, nb, Hk, bs, D, dev)
    # a few tokens outgrow what their block held
    big = torch.where(torch.rand((T, 1, 1), generator=g, device=dev) < 0.2, 6.0, 1.0)
    s["k"] = (_rows(g, (T, Hk, D), dev, "k") * big).to(dtype)
    s["v"] = (_rows(g, (T, Hk, D), dev, "v") * big).to(dtype)
    # every token from the first one of the first block written
    near = [torch.arange(n // bs * bs, n + new, device=dev) for n in lens]
    s["read"] = torch.cat([_slots_at(table, b, t, bs) for b, t in enumerate(near)])
    s["k_out"] = torch.empty((s["read"].numel(), Hk, D), dtype=dtype, device=dev)
    s["v_out"] = torch.empty_like(s["k_out"])


def _prepare_read(case, s, g, dev, bs):
    T, Hk, D, dtype = case["T"], case["Hk"], case["D"], _DTYPES[case["dtype"]]
    nb = _blocks(T, bs) + 1
    perm = torch.randperm(nb, generator=g, device=dev)
    t = torch.arange(T, device=dev)
    s["read"] = (perm[t // bs] * bs + t % bs).to(torch.int32)
    s["kc"], s["vc"], s["scales"] = _cache8(g, nb, Hk, bs, D, dev)
    s["k_out"] = torch.empty((T, Hk, D), dtype=dtype, device=dev)
    s["v_out"] = torch.empty_like(s["k_out"])


def _prepare_decode(case, s, g, dev, bs):
    B, H, Hk, D, dtype = case["B"], case["H"], case["Hk"], case["D"], _DTYPES[case["dtype"]]
    base = _lengths(case)
    lens = [base[i] for i in torch.randperm(B, generator=g, device=dev).tolist()]
    need = sum(_blocks(n, bs) for n in lens)
    nb = need + need // 10 + 1
    perm = torch.randperm(nb, generator=g, device=dev)
    s["max_len"] = max(lens)
    s["table"], _ = _table(perm, lens, max(1, _blocks(max(lens), bs)), bs, dev)
    s["lens"] = _i32(lens, dev)
    s["kc"], s["vc"], s["scales"] = _cache8(g, nb, Hk, bs, D, dev)
    s["scale"] = D ** -0.5
    s["q"] = (torch.randn((B, H, D), generator=g, device=dev) * case["gain"]).to(dtype)
    s["out"] = torch.empty_like(s["q"])


# ---------------------------------------------------------------------------- one pass

def run(s):
    kind = s["case"]["kind"]
    if own:
        return _own(s, kind)
    return {"layout": _plain_layout, "rotary": _plain_rotary, "write": _plain_write, "read": _plain_read,
            "decode": _plain_decode}[kind](s)


def _layout_out(s):
    return s["table"], s["lens_2"], s["num_free_2"], s["free"], s["start"], s["slots"], s["positions"]


def _own(s, kind):
    import paged_kv_cache_261_gb300 as pa
    case = s["case"]
    if kind == "layout":
        pa.paged_blocks_release(s["table"], s["lens"], s["done"], s["free"], s["num_free"], case["bs"],
                                new_context_lens=s["lens_1"], new_num_free=s["num_free_1"])
        pa.paged_blocks_append(s["table"], s["lens_1"], s["new"], s["free"], s["num_free_1"], s["start"], s["slots"],
                               s["positions"], case["bs"], s["nb"], new_context_lens=s["lens_2"],
                               new_num_free=s["num_free_2"])
        return _layout_out(s)
    if kind == "rotary":
        how = {"factor": s["factor"], "interleaved": case["pairs"] == "interleaved"}
        if case["store"]:
            pa.paged_kv_write_rotary(s["q_out"], s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["slots"],
                                     s["kc"], s["vc"], **how)
            return s["q_out"], s["kc"], s["vc"]
        pa.rotary_embedding(s["q_out"], s["k_out"], s["q"], s["k"], s["positions"], s["inv_freq"], **how)
        return s["q_out"], s["k_out"]
    if kind == "decode":
        pa.paged_attention_decode_fp8_block(s["out"], s["q"], s["kc"], s["vc"], s["scales"], s["table"], s["lens"],
                                            s["scale"], max_context_len=s["max_len"])
        return s["out"]
    if kind == "write":
        pa.paged_kv_write_fp8_block(s["k"], s["v"], s["slots"], s["kc"], s["vc"], s["scales"])
    pa.paged_kv_read_fp8_block(s["k_out"], s["v_out"], s["read"], s["kc"], s["vc"], s["scales"])
    return (s["k_out"], s["v_out"], s["scales"]) if kind == "write" else (s["k_out"], s["v_out"])


def _plain_layout(s):
    bs, table, free = s["case"]["bs"], s["table"], s["free"]
    width, dev = table.shape[1], table.device
    j = torch.arange(width, device=dev)
    # the finished requests' blocks go back, in order
    c, nf = s["lens"].long(), s["num_free"].long()
    back = torch.where(s["done"], (c + bs - 1) // bs, torch.zeros_like(c))
    before = torch.cumsum(back, 0) - back
    at = (nf + before)[:, None] + j
    live = j < back[:, None]
    free[at[live]] = table[live]
    c = torch.where(s["done"], torch.zeros_like(c), c)
    nf = nf + back.sum()
    s["lens_1"].copy_(c)
    s["num_free_1"].copy_(nf)
    # the new tokens take blocks off the end of the list
    n = s["new"].long()
    held = (c + bs - 1) // bs
    need = (c + n + bs - 1) // bs - held
    upto = torch.cumsum(need, 0)
    fits = (need == 0) | (upto <= nf)
    live = (j >= held[:, None]) & (j < (held + need)[:, None]) & fits[:, None]
    at = nf - 1 - ((upto - need - held)[:, None] + j)
    table[live] = free[at[live]]
    taken = torch.where(fits, need, torch.zeros_like(need)).sum()
    s["num_free_2"].copy_(nf - taken)
    s["lens_2"].copy_(torch.where(fits, c + n, c))
    s["start"][1:] = torch.cumsum(n, 0).to(torch.int32)
    t = torch.arange(s["slots"].numel(), device=dev)
    start = s["start"].long()
    b = torch.searchsorted(start[1:].contiguous(), t, right=True).clamp(max=n.numel() - 1)
    pos = c[b] + t - start[b]
    ok = (t < start[-1]) & fits[b]
    pos = torch.where(ok, pos, torch.zeros_like(pos))
    slot = table[b, pos // bs].long() * bs + pos % bs
    s["slots"].copy_(torch.where(ok, slot, torch.full_like(slot, -1)))
    s["positions"].copy_(pos)
    return _layout_out(s)


def _rotate(x, cos, sin, pairs):
    """x [T, heads, D] in float32 with its first 2 * cos.shape[-1] channels rotated."""
    half = cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    y = x.clone()
    if pairs == "half":
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half] = a * cos - b * sin
        y[..., half:2 * half] = b * cos + a * sin
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2] = a * cos - b * sin
        y[..., 1:2 * half:2] = b * cos + a * sin
    return y


def _plain_rotary(s):
    case = s["case"]
    angle = s["positions"].double()[:, None] * s["inv_freq"]          # far positions need 64 bits
    cos, sin = (angle.cos() * s["factor"]).float(), (angle.sin() * s["factor"]).float()
    s["q_out"].copy_(_rotate(s["q"].float(), cos, sin, case["pairs"]))
    k = _rotate(s["k"].float(), cos, sin, case["pairs"]).to(s["k"].dtype)
    if not case["store"]:
        s["k_out"].copy_(k)
        return s["q_out"], s["k_out"]
    live = s["slots"] >= 0
    slots = s["slots"].long()[live]
    s["kc"].view(-1, case["Hk"], case["D"])[slots] = k[live]
    s["vc"].view(-1, case["Hk"], case["D"])[slots] = s["v"][live]
    return s["q_out"], s["kc"], s["vc"]


def _plain_write(s):
    case = s["case"]
    bs, Hk = case["bs"], case["Hk"]
    nb = s["kc"].shape[0]
    live = s["slots"] >= 0
    slots = s["slots"].long()[live]
    block, off = slots // bs, slots % bs
    new = torch.zeros(nb, dtype=torch.bool, device=slots.device)
    new[block[off == 0]] = True                                       # blocks that start anew
    hit = torch.zeros_like(new)
    hit[block] = True
    hit = hit.nonzero().flatten()
    for j, (x, cache) in enumerate((("k", "kc"), ("v", "vc"))):
        x = s[x][live].float()
        amax = torch.zeros((nb, Hk), device=x.device).index_reduce_(0, block, x.abs().amax(-1), "amax")
        old = s["scales"][hit, :, j]
        want = _scale_for(amax[hit])
        scale = torch.where(new[hit][:, None], want, torch.maximum(old, want))
        codes = s[cache][hit]
        again = _codes(_values(codes) * torch.where(new[hit][:, None], torch.ones_like(old), old / scale)[..., None, None])
        s[cache][hit] = torch.where((new[hit][:, None] | (scale == old))[..., None, None], codes, again)
        s["scales"][hit, :, j] = scale
        s[cache][block, :, off] = _codes(x / s["scales"][block, :, j][..., None])
    k, v = _plain_read(s)
    return k, v, s["scales"]


def _read8(s, slots):
    """K and V values in float32 at `slots` [n]: two [n, Hk, D]."""
    bs = s["case"]["bs"]
    block, off = slots // bs, slots % bs
    scale = s["scales"][block]
    return (_values(s["kc"][block, :, off]) * scale[:, :, 0:1], _values(s["vc"][block, :, off]) * scale[:, :, 1:2])


def _plain_read(s):
    k, v = _read8(s, s["read"].long())
    s["k_out"].copy_(k)
    s["v_out"].copy_(v)
    return s["k_out"], s["v_out"]


def _plain_decode(s):
    case = s["case"]
    bs, Hk, n = case["bs"], case["Hk"], s["max_len"]
    B, H, D = s["q"].shape
    t = torch.arange(n, device=s["q"].device)
    slots = s["table"].long().clamp(min=0)[:, t // bs] * bs + t % bs
    k, v = _read8(s, slots.flatten())
    k = k.view(B, n, Hk, D).permute(0, 2, 3, 1)                       # [B, Hk, D, n]
    v = v.view(B, n, Hk, D).permute(0, 2, 1, 3)                       # [B, Hk, n, D]
    q = s["q"].float().view(B, Hk, H // Hk, D)
    x = torch.matmul(q, k) * s["scale"]
    live = (t < s["lens"][:, None])[:, None, None]                    # a context of no tokens has no weights
    e = torch.where(live, torch.exp(x - x.masked_fill(~live, -3.0e38).amax(-1, keepdim=True)), torch.zeros_like(x))
    w = e / e.sum(-1, keepdim=True).clamp(min=1e-30)
    s["out"].copy_(torch.matmul(w, v).reshape(B, H, D))
    return s["out"]


# ---------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"layout": _exact_layout, "rotary": _exact_rotary, "write": _exact_write, "read": _exact_read,
            "decode": _exact_decode}[case["kind"]](s, case)


def _exact_layout(s, case):
    bs, dev = case["bs"], s["table"].device
    table, free = s["table"].tolist(), s["free"].tolist()
    lens, new, done, nf = s["lens"].tolist(), s["new"].tolist(), s["done"].tolist(), int(s["num_free"])
    for b, d in enumerate(done):
        if d:
            for j in range(_blocks(lens[b], bs)):
                free[nf] = table[b][j]
                nf += 1
            lens[b] = 0
    start, slots, positions, left, dry = [0], [], [], nf, False
    for b, n in enumerate(new):
        c = lens[b]
        need = _blocks(c + n, bs) - _blocks(c, bs)
        start.append(start[-1] + n)
        dry = dry or need > left
        if need and dry:                          # from the first request that finds too few, none is served
            slots += [-1] * n
            positions += [0] * n
            continue
        for j in range(need):
            left -= 1
            table[b][_blocks(c, bs) + j] = free[left]
        for i in range(c, c + n):
            slots.append(table[b][i // bs] * bs + i % bs)
            positions.append(i)
        lens[b] = c + n
    rest = s["slots"].numel() - len(slots)
    return tuple(_i32(x, dev) for x in (table, lens, [left], free, start, slots + [-1] * rest, positions + [0] * rest))


def _exact_rotary(s, case):
    half = case["rd"] // 2
    f = torch.tensor(_frequencies(case)[0], dtype=torch.float64, device=s["q"].device)
    z = torch.polar(torch.full_like(f, s["factor"]).expand(case["T"], half).contiguous(),
                    s["positions"].double()[:, None] * f)[:, None]
    out = []
    for x in (s["q"].double(), s["k"].double()):
        head = x[..., :2 * half]
        pair = head.unflatten(-1, (2, half)).transpose(-1, -2) if case["pairs"] == "half" else head.unflatten(-1, (half, 2))
        turned = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
        turned = turned.transpose(-1, -2) if case["pairs"] == "half" else turned
        out.append(torch.cat((turned.reshape(head.shape), x[..., 2 * half:]), -1))
    if not case["store"]:
        return tuple(out)
    kc, vc = s["kc"].double(), s["vc"].double()
    for t in torch.arange(case["T"] - case["pad"], device=kc.device).split(1024):
        b, o = torch.div(s["slots"][t].long(), case["bs"], rounding_mode="floor"), s["slots"][t].long() % case["bs"]
        kc[b, o] = out[1][t]
        vc[b, o] = s["v"][t].double()
    return out[0], kc, vc


def _pow2(e):
    """2^e in 64 bits, of whole numbers e."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _grid64(x):
    """x rounded to the nearest E4M3 value, ties to even, in 64 bits; |x| <= 448."""
    step = _pow2((torch.frexp(x).exponent - 1).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _e4m3(codes):
    """The values of E4M3 codes in 64 bits, from their fields."""
    c = codes.long()
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * _pow2(e - 10))
    return torch.where(c >= 128, -v, v)


def _exact_read(s, case):
    bs = case["bs"]
    out = [torch.empty(s["k_out"].shape, dtype=torch.float64, device=s["k_out"].device) for _ in range(2)]
    for t in torch.arange(s["read"].numel(), device=s["read"].device).split(16384):
        slot = s["read"][t].long()
        b, o = torch.div(slot, bs, rounding_mode="floor"), slot.remainder(bs)
        for j, c in enumerate(("kc", "vc")):
            out[j][t] = _e4m3(s[c][b, :, o]) * s["scales"][b, :, j].double()[..., None]
    return tuple(out)


def _exact_write(s, case):
    bs, scales = case["bs"], s["scales"].double()
    held = {}                                                         # block -> its values, K and V
    slots = s["slots"].tolist()
    by_block = {}
    for t, slot in enumerate(slots):
        if slot >= 0:
            by_block.setdefault(slot // bs, []).append((t, slot % bs))
    if len(by_block) > 4096:
        return None
    for b, tokens in by_block.items():
        at = torch.tensor([t for t, _ in tokens], device=scales.device)
        off = torch.tensor([o for _, o in tokens], device=scales.device)
        fresh = any(o == 0 for _, o in tokens)
        both = []
        for j, (x, c) in enumerate((("k", "kc"), ("v", "vc"))):
            x = s[x][at].double().transpose(0, 1)                     # [Hk, tokens, D]
            top = x.abs().amax((1, 2))
            at_most = torch.arange(-100, 121, device=top.device)      # the first of the scales that suffices
            want = _pow2(at_most[(448 * _pow2(at_most) < top[:, None]).sum(1)])
            old = scales[b, :, j]
            scale = want if fresh else torch.maximum(old, want)
            values = _e4m3(s[c][b]) * old[:, None, None]              # [Hk, bs, D]
            if not fresh:
                values = torch.where((scale > old)[:, None, None], _grid64(values / scale[:, None, None]) *
                                     scale[:, None, None], values)
            values[:, off] = _grid64(x / scale[:, None, None]) * scale[:, None, None]
            scales[b, :, j] = scale
            both.append(values)
        held[b] = both
    blocks = sorted(held)
    where = torch.full((s["kc"].shape[0],), -1, device=scales.device, dtype=torch.long)
    where[blocks] = torch.arange(len(blocks), device=scales.device)
    slot = s["read"].long()
    out = [torch.stack([held[b][j] for b in blocks])[where[slot // bs], :, slot % bs] for j in range(2)]
    return out[0], out[1], scales


def _exact_decode(s, case):
    B, H, D = s["q"].shape
    bs, Hk = case["bs"], case["Hk"]
    G = H // Hk
    out = torch.zeros((B, H, D), dtype=torch.float64, device=s["q"].device)
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        blk = s["table"][b, :_blocks(n, bs)].long()
        for h in range(Hk):
            k, v = ((_e4m3(s[c][blk, h]) * s["scales"][blk, h, j].double()[:, None, None]).reshape(-1, D)[:n]
                    for j, c in enumerate(("kc", "vc")))
            w = torch.softmax(k @ s["q"][b, h * G:(h + 1) * G].double().t() * s["scale"], 0)   # [n, G]
            out[b, h * G:(h + 1) * G] = w.t() @ v
    return out
