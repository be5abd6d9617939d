"""Measured cases of the positions-and-cache operators: rotary positions with several axes, appending to the
8-bit block cache, and attention over that cache.

`run` computes an operator in its plain form (elementary torch operations), or, where `own` is true, through
this library's entry points.  Both work on the same tensors, which `prepare` makes from a case and a seed.

The cache (one layer of one model):
  k_pages, v_pages  e4m3    [P, H, 64, d]     closed blocks: 64 tokens of one sequence, every key/value head
  k_scale, v_scale  float32 [P, H]            one power of two per block and head; a value is code * scale
  k_tail, v_tail    bf16    [B, 2, H, 64, d]  the open block of each sequence, in one of two slots
  page_table        int32   [B, blocks]       the page of each closed block of a sequence
  seq               int32   [B, 2]            tokens held, and the tail slot that holds the open block
"""
import math

import torch

own = False

BLOCK = 64
E4M3_MAX = 448.0
MIN_EXPONENT = -100   # of a block's scale


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # One 480p clip's queries and keys turned before the sparse branch (20 x 30 x 52 latent).
        dict(name="rope_480p", op="rope", dtype="bfloat16", B=1, H=12, Hk=12, N=31200, d=128, Hh=30, Wh=52,
             s0=44, s1=42, s2=42, far=0, pairing="adjacent", layout="heads", backward=False),
        # The gradient of one 720p clip's queries, 40 heads (28 x 45 x 80 latent).
        dict(name="rope_720p_backward", op="rope", dtype="bfloat16", B=1, H=40, Hk=0, N=100800, d=128, Hh=45, Wh=80,
             s0=44, s1=42, s2=42, far=0, pairing="adjacent", layout="heads", backward=True),
        # Single tokens of eight sequences at far positions, grouped key heads: latency.
        dict(name="rope_token", op="rope", dtype="bfloat16", B=8, H=40, Hk=8, N=1, d=128, Hh=0, Wh=0,
             s0=44, s1=42, s2=42, far=1 << 20, pairing="adjacent", layout="heads", backward=False),
        # Float32 training on images (two axes), token-major tensors as a projection writes them, odd length.
        dict(name="rope_image_f32_backward", op="rope", dtype="float32", B=3, H=12, Hk=12, N=4097, d=64, Hh=0, Wh=0,
             s0=0, s1=32, s2=32, far=4096, pairing="halves", layout="tokens", backward=True),
        # Three latent frames of 480p written behind three chunks: video generated chunk by chunk.
        dict(name="append_chunk", op="append", B=1, H=12, N=4680, d=128, past=14040, stagger=0, pad=0, Hh=30, Wh=52),
        # One token of each of 16 sequences of different lengths: latency.
        dict(name="append_token", op="append", B=16, H=12, N=1, d=128, past=2111, stagger=61, pad=0, Hh=30, Wh=52),
        # A padded batch of 720p chunks with 40 heads, given positions.
        dict(name="append_ragged", op="append", B=4, H=40, N=3600, d=128, past=7777, stagger=1901, pad=641, Hh=0, Wh=0),
        # One query token of one sequence over a whole 480p clip: reads the cache once.
        dict(name="attn_token", op="attn", B=1, Hq=12, H=12, N=1, d=128, past=31200, stagger=0, pad=0, frame=0, window=-1),
        # A batch of single tokens, five query heads to a key head, ragged lengths.
        dict(name="attn_token_grouped", op="attn", B=16, Hq=40, H=8, N=1, d=128, past=16001, stagger=977, pad=0, frame=1,
             window=-1),
        # A small layer: 16 query tokens, short odd lengths (latency).
        dict(name="attn_small", op="attn", B=2, Hq=2, H=2, N=16, d=64, past=1000, stagger=371, pad=3, frame=1, window=-1),
        # Three latent frames of 480p, each seeing its own frame and every earlier one.
        dict(name="attn_chunk", op="attn", B=1, Hq=12, H=12, N=4680, d=128, past=18720, stagger=0, pad=0, frame=1560,
             window=-1),
        # One latent frame over a whole 720p clip (8 heads).
        dict(name="attn_frame_720p", op="attn", B=1, Hq=8, H=8, N=3600, d=128, past=100800, stagger=0, pad=0, frame=0,
             window=-1),
    ]


def _span(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn"])
    d = rng.choice([64, 128])
    if op == "rope":
        N = _span(rng, 1, 100800)
        H = rng.choice([1, 2, 8, 12, 40])
        B = _span(rng, 1, max(1, min(16, 40 * 100800 // (H * N))))
        grid = rng.random() < 0.5
        dy = 2 * (d // 6)
        split = (d - 2 * dy, dy, dy) if grid else rng.choice([(d - 2 * dy, dy, dy), (0, d // 2, d // 2), (d, 0, 0)])
        Hh, Wh = (rng.randint(1, 60), rng.randint(1, 90)) if grid else (0, 0)
        dtype = rng.choice(["bfloat16", "bfloat16", "float16", "float32"]) if B * H * N * d < 1 << 27 else "bfloat16"
        return dict(op=op, dtype=dtype, B=B, H=H, Hk=rng.choice([0, 1, H]) if B * H * N * d < 1 << 27 else 0, N=N, d=d,
                    Hh=Hh, Wh=Wh, s0=split[0], s1=split[1], s2=split[2], far=0 if grid else _span(rng, 16, 1 << 24),
                    pairing=rng.choice(["adjacent", "halves"]), layout=rng.choice(["heads", "tokens"]),
                    backward=rng.random() < 0.5)
    B = _span(rng, 1, 16)
    past = _span(rng, 1, 40000)
    stagger = rng.randint(0, max(0, past // B))
    if op == "append":
        N = _span(rng, 1, 4680)
        H = rng.choice([h for h in (1, 2, 8, 12, 40) if B * h * N <= 4 * 40 * 3600] or [1])
        Hh, Wh = (rng.randint(1, 60), rng.randint(1, 90)) if rng.random() < 0.5 else (0, 0)
        return dict(op=op, B=B, H=H, N=N, d=d, past=past, stagger=stagger, pad=rng.randint(0, max(0, N // B)), Hh=Hh, Wh=Wh)
    N = _span(rng, 1, min(4680, past))
    most = 8 * 3600 * 100800
    heads = [(q, h) for q, h in ((1, 1), (2, 2), (8, 8), (12, 12), (12, 3), (40, 8), (40, 40)) if B * q * N * past <= most // 4]
    Hq, H = rng.choice(heads or [(1, 1)])
    while B > 1 and B * Hq * N * past > most // 4:
        B -= 1
    frame = rng.choice([0, 1, rng.randint(1, 1600)])
    return dict(op=op, B=B, Hq=Hq, H=H, N=N, d=d, past=past, stagger=min(stagger, past // B),
                pad=rng.randint(0, max(0, N // B)), frame=frame, window=rng.choice([-1, -1, _span(rng, 1, 20000)]))


def _lengths(case):
    """Tokens held by each sequence (before an append; with the queries' own keys for an attention)."""
    return [max(0, case["past"] - b * case["stagger"]) for b in range(case["B"])]


def _counts(case):
    """Valid tokens of each sequence's row of the batch."""
    return [max(0, case["N"] - b * case["pad"]) for b in range(case["B"])]


# ----------------------------------------------------------------- inputs --
def _codes(x):
    """Blocks [.., 64, d] as e4m3 codes and their power-of-two scales [..]: the smallest that keeps every code
    within e4m3's range."""
    part, e = torch.frexp(x.abs().amax(dim=(-2, -1)).float() / E4M3_MAX)
    e = e - (part == 0.5).to(e.dtype)
    scale = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e.clamp(min=MIN_EXPONENT))
    return (x.float() / scale[..., None, None]).to(torch.float8_e4m3fn), scale


def _cache(case, g, heads, lens, grow):
    """A cache that holds `lens` tokens of each sequence and has room for `grow` more, its pages in random order."""
    dev, B, d = "cuda", case["B"], case["d"]
    blocks = max(1, (max(lens) + grow + BLOCK - 1) // BLOCK)
    P = B * blocks + 3
    table = torch.randperm(P, generator=g, device=dev)[: B * blocks].reshape(B, blocks).to(torch.int32)
    c = {"page_table": table}
    for name in ("k", "v"):
        # Channels of different size, as keys have them.
        size = torch.exp(0.5 * torch.randn(heads, 1, d, generator=g, device=dev))
        x = torch.randn(P, heads, BLOCK, d, generator=g, device=dev)
        c[name + "_pages"], c[name + "_scale"] = _codes(x.mul_(size))
        c[name + "_tail"] = (torch.randn(B, 2, heads, BLOCK, d, generator=g, device=dev) * size).to(torch.bfloat16)
    slots = torch.randint(0, 2, (B,), generator=g, device=dev)
    c["seq"] = torch.stack([torch.tensor(lens, device=dev), slots], dim=1).to(torch.int32)
    return c


def _handle(c):
    """The library's object for a cache of these tensors, as a program keeps one beside its layer."""
    import sparse_linear_hybrid_top_b200 as salad
    return salad.BlockCache(c["k_pages"], c["v_pages"], c["k_scale"], c["v_scale"], c["k_tail"], c["v_tail"],
                            c["page_table"])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    B, N, d, op = case["B"], case["N"], case["d"], case["op"]

    def rand(heads, dtype, layout="heads"):
        if layout == "tokens":
            return torch.randn(B, N, heads, d, generator=g, device="cuda").to(dtype).transpose(1, 2)
        return torch.randn(B, heads, N, d, generator=g, device="cuda").to(dtype)

    def positions(far):
        return torch.randint(0, far + 1, (B, N, 3), generator=g, device="cuda", dtype=torch.int32)

    s = {"case": case}
    if op == "rope":
        dtype = getattr(torch, case["dtype"])
        s["q"] = rand(case["H"], dtype, case["layout"])
        s["k"] = rand(case["Hk"], dtype, case["layout"]) if case["Hk"] else None
        s["positions"] = positions(case["far"]) if not case["Hh"] else None
        return s
    lens, counts = _lengths(case), _counts(case)
    s["counts"] = torch.tensor(counts, dtype=torch.int32, device="cuda") if case["pad"] else None
    if op == "append":
        s["cache"] = _cache(case, g, case["H"], lens, N)
        s["k"], s["v"] = rand(case["H"], torch.bfloat16), rand(case["H"], torch.bfloat16)
        s["positions"] = positions(4096) if not case["Hh"] else None
        s["seq_out"] = torch.zeros(B, 2, dtype=torch.int32, device="cuda")
    else:
        s["cache"] = _cache(case, g, case["H"], lens, 0)
        s["q"] = rand(case["Hq"], torch.bfloat16)
        # Rows behind a sequence's last query stay as they are: zeros here.
        s["o"] = torch.zeros(B, case["Hq"], N, d, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.zeros(B, case["Hq"], N, dtype=torch.float32, device="cuda")
    if own:
        s["handle"] = _handle(s["cache"])
    return s


# ------------------------------------------------------------- plain forms --
def _split(case):
    d = case["d"]
    dy = 2 * (d // 6)
    return (case["s0"], case["s1"], case["s2"]) if "s0" in case else (d - 2 * dy, dy, dy)


def _grid_positions(p, Hh, Wh):
    return torch.stack([p // (Hh * Wh), p // Wh % Hh, p % Wh], dim=-1)


def _turn(x, pos, split, pairing, sign):
    """x [B, H, N, d] float32, each channel pair turned by its angle; pos [B or 1, N, 3]."""
    dev = x.device
    rate = torch.cat([10000.0 ** (-2.0 * torch.arange(s // 2, device=dev, dtype=torch.float64) / max(s, 1)) for s in split])
    axis = torch.repeat_interleave(torch.arange(3, device=dev), torch.tensor([s // 2 for s in split], device=dev),
                                   output_size=rate.numel())
    angle = pos[..., axis].double() * rate                       # [B, N, d/2]
    c, s = torch.cos(angle).float()[:, None], (sign * torch.sin(angle)).float()[:, None]
    if pairing == "adjacent":
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * s, a * s + b * c], dim=-1).flatten(-2)
    a, b = x.chunk(2, dim=-1)
    return torch.cat([a * c - b * s, a * s + b * c], dim=-1)


def _plain_rope(s):
    case = s["case"]
    pos = s["positions"]
    if pos is None:
        pos = _grid_positions(torch.arange(case["N"], device="cuda"), case["Hh"], case["Wh"])[None]
    sign = -1.0 if case["backward"] else 1.0
    return [_turn(t.float(), pos, _split(case), case["pairing"], sign).to(t.dtype)
            for t in (s["q"], s["k"]) if t is not None]


def _plain_append(s):
    case, c = s["case"], s["cache"]
    B, H, N, d = s["k"].shape
    dev = s["k"].device
    n = torch.full((B,), N, device=dev) if s["counts"] is None else s["counts"].long()
    length, slot = c["seq"][:, 0].long(), c["seq"][:, 1].long()
    first, last = length // BLOCK, (length + n) // BLOCK          # open block before and after
    slot_out = torch.where(first == last, slot, 1 - slot)
    pos = s["positions"]
    if pos is None:
        pos = _grid_positions(length[:, None] + torch.arange(N, device=dev), case["Hh"], case["Wh"])
    k = _turn(s["k"].float(), pos, _split(case), "adjacent", 1.0).to(torch.bfloat16)
    # Every block that the call touches, from its own rows and the open block's.
    span = (N + BLOCK - 1) // BLOCK + 1
    row = torch.arange(span * BLOCK, device=dev)
    token = row - (length % BLOCK)[:, None]                       # [B, span * 64], in this call
    seq = torch.arange(B, device=dev)
    new = (token >= 0) & (token < n[:, None])
    block = first[:, None] + torch.arange(span, device=dev)      # [B, span]
    closed = block < last[:, None]
    which, at = closed.nonzero(as_tuple=True)
    page = c["page_table"][which, block[which, at]].long()
    bt, rt = (new & (block.repeat_interleave(BLOCK, 1) == last[:, None])).nonzero(as_tuple=True)
    for name, x in (("k", k), ("v", s["v"])):
        tail = c[name + "_tail"]
        got = torch.gather(x, 2, token.clamp(0, N - 1)[:, None, :, None].expand(B, H, span * BLOCK, d))
        old = tail[seq, slot].repeat(1, 1, span, 1)
        rows = torch.where(new[:, None, :, None], got, old).reshape(B, H, span, BLOCK, d)
        codes, scale = _codes(rows[which, :, at])
        c[name + "_pages"].view(torch.uint8)[page] = codes.view(torch.uint8)
        c[name + "_scale"][page] = scale
        tail[bt, slot_out[bt], :, rt % BLOCK] = rows.reshape(B, H, span * BLOCK, d)[bt, :, rt]
    s["seq_out"].copy_(torch.stack([length + n, slot_out], dim=1))
    return _append_outputs(s)


def _append_outputs(s):
    c = s["cache"]
    return {"seq": s["seq_out"], **{x: c[x] for x in ("k_pages", "v_pages", "k_scale", "v_scale", "k_tail", "v_tail")}}


def _held(c, name, length, slot, blocks):
    """The cache's keys or values as float32 [B, H, blocks * 64, d]; 0 behind the last token."""
    B = length.numel()
    dev = length.device
    page = c["page_table"][:, :blocks].long()
    x = c[name + "_pages"][page].float() * c[name + "_scale"][page][..., None, None]      # [B, blocks, H, 64, d]
    tail = c[name + "_tail"][torch.arange(B, device=dev), slot].float()[:, None]
    block = torch.arange(blocks, device=dev)
    x = torch.where((block == (length // BLOCK)[:, None])[:, :, None, None, None], tail, x)
    x = x.permute(0, 2, 1, 3, 4).flatten(2, 3)
    held = torch.arange(blocks * BLOCK, device=dev) < length[:, None]
    return torch.where(held[:, None, :, None], x, torch.zeros((), device=dev))


def _visible(case, length, n, keys):
    """Which keys each query row sees: [B, N, keys]."""
    dev = length.device
    i = torch.arange(case["N"], device=dev)
    j = torch.arange(keys, device=dev)
    start = (length - n)[:, None]
    if case["frame"]:
        group = torch.div(start + i, case["frame"], rounding_mode="floor") * case["frame"]
        end = torch.minimum(group + case["frame"], length[:, None])
    else:
        group = start.expand(-1, case["N"])
        end = length[:, None].expand(-1, case["N"])
    low = group - case["window"] if case["window"] >= 0 else torch.zeros_like(group)
    return (j >= low[..., None]) & (j < end[..., None])


def _plain_attn(s):
    case, c, q = s["case"], s["cache"], s["q"]
    B, Hq, N, d = q.shape
    H, dev = case["H"], q.device
    length, slot = c["seq"][:, 0].long(), c["seq"][:, 1].long()
    n = torch.full((B,), N, device=dev) if s["counts"] is None else s["counts"].long()
    blocks = c["page_table"].shape[1]
    k, v = _held(c, "k", length, slot, blocks), _held(c, "v", length, slot, blocks)
    x = (q.float() / math.sqrt(d)).reshape(B, H, Hq // H * N, d) @ k.transpose(-1, -2)
    x = x.reshape(B, H, Hq // H, N, -1)
    see = _visible(case, length, n, blocks * BLOCK)[:, None, None]
    x = x.masked_fill_(~see, -math.inf)
    m = x.amax(dim=-1, keepdim=True)
    p = x.sub_(m.clamp(min=-1e30)).exp_()
    total = p.sum(dim=-1, keepdim=True)
    o = (p.reshape(B, H, Hq // H * N, -1) @ v).reshape(B, H, Hq // H, N, d) / torch.where(total > 0, total, 1.0)
    lse = (m + torch.log(total)).reshape(B, Hq, N)
    valid = (torch.arange(N, device=dev) < n[:, None])[:, None]
    s["o"].copy_(torch.where(valid[..., None], o.reshape(B, Hq, N, d).to(q.dtype), s["o"]))
    s["lse"].copy_(torch.where(valid, lse, s["lse"]))
    return {"o": s["o"], "lse": s["lse"]}


def run(state):
    case = state["case"]
    if own:
        import sparse_linear_hybrid_top_b200 as salad
        if case["op"] == "rope":
            call = salad.rope_backward if case["backward"] else salad.rope
            kw = {"positions": state["positions"]} if state["positions"] is not None else {"grid": (case["Hh"], case["Wh"])}
            out = call(state["q"], state["k"], split=_split(case), pairing=case["pairing"], **kw)
            return [t for t in out if t is not None] if isinstance(out, tuple) else [out]
        if case["op"] == "append":
            kw = {"positions": state["positions"]} if state["positions"] is not None else {"grid": (case["Hh"], case["Wh"])}
            salad.cache_append(state["handle"], state["k"], state["v"], state["cache"]["seq"], counts=state["counts"],
                               seq_out=state["seq_out"], **kw)
            return _append_outputs(state)
        salad.cache_attn(state["handle"], state["q"], state["cache"]["seq"], counts=state["counts"], frame=case["frame"],
                         window=case["window"], o=state["o"], lse=state["lse"])
        return {"o": state["o"], "lse": state["lse"]}
    return {"rope": _plain_rope, "append": _plain_append, "attn": _plain_attn}[case["op"]](state)


# ------------------------------------------------------------------- work --
def work(case):
    d, B, N = case["d"], case["B"], case["N"]
    if case["op"] == "rope":
        elements = B * (case["H"] + case["Hk"]) * N * d
        width = 4 if case["dtype"] == "float32" else 2
        return {"bytes": 2 * elements * width + (0 if case["Hh"] else B * N * 12), "flops": 3 * elements}
    lens, counts = _lengths(case), _counts(case)
    if case["op"] == "append":
        bytes_, H = 0, case["H"]
        for length, n in zip(lens, counts):
            first, last = length // BLOCK, (length + n) // BLOCK
            row = 2 * H * d                                       # one token's keys and values, in elements
            bytes_ += n * row * 2 + (0 if case["Hh"] else 12 * n) # read the new tokens
            if last > first:
                bytes_ += (length % BLOCK) * row * 2              # read the open block that closes
                bytes_ += (last - first) * (BLOCK * row + 8 * H)  # write closed blocks and their scales
                bytes_ += (length + n) % BLOCK * row * 2          # write the new open block
            else:
                bytes_ += n * row * 2
            bytes_ += 16
        return {"bytes": bytes_, "flops": 3 * sum(counts) * H * d}
    Hq, H, frame, window = case["Hq"], case["H"], case["frame"], case["window"]
    bytes_ = pairs = 0
    for length, n in zip(lens, counts):
        start = length - n
        groups = [(start, length)] * n if not frame else \
            [((start + i) // frame * frame, min(length, (start + i) // frame * frame + frame)) for i in range(n)]
        spans = [(max(0, a - window) if window >= 0 else 0, e) for a, e in groups]
        pairs += sum(max(0, e - a) for a, e in spans)
        lo, hi = min((a for a, e in spans if e > a), default=0), max((e for a, e in spans if e > a), default=0)
        closed = max(0, min(hi, length // BLOCK * BLOCK) - lo)
        bytes_ += 2 * H * d * (closed + 2 * max(0, hi - lo - closed)) + (hi - lo + BLOCK - 1) // BLOCK * 8 * H
        bytes_ += n * Hq * (4 * d + 4)
    return {"bytes": bytes_, "flops": 4 * d * Hq * pairs}


# ------------------------------------------------------------- definitions --
# The operators again from their definitions in 64 bits, one sequence and head at a time where that is clearer.
def _exact_turn(x, pos, split, pairing, sign):
    out = x.clone()
    d = x.shape[-1]
    m = 0
    for axis, size in enumerate(split):
        for i in range(size // 2):
            a = sign * pos[:, axis].double() * math.exp(-2.0 * i / size * math.log(10000.0))
            u, w = (2 * m, 2 * m + 1) if pairing == "adjacent" else (m, m + d // 2)
            out[..., u] = x[..., u] * torch.cos(a) - x[..., w] * torch.sin(a)
            out[..., w] = x[..., u] * torch.sin(a) + x[..., w] * torch.cos(a)
            m += 1
    return out


def _exact_codes(x):
    """What e4m3 holds of one head's block: values without the scale, and the scale."""
    top = float(x.abs().max())
    e = MIN_EXPONENT
    if top > 0:
        e = max(e, math.frexp(top / E4M3_MAX)[1] - (1 if math.frexp(top / E4M3_MAX)[0] == 0.5 else 0))
    y = x / 2.0 ** e
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step, 2.0 ** e


def exact(case, seed):
    s = prepare(case, seed)
    B, N, d = case["B"], case["N"], case["d"]
    if case["op"] == "rope":
        out = []
        for t in (s["q"], s["k"]):
            if t is None:
                continue
            r = torch.empty(t.shape, dtype=torch.float64, device=t.device)
            for b in range(B):
                if s["positions"] is not None:
                    pos = s["positions"][b]
                else:
                    n = torch.arange(N, device=t.device)
                    x, y = n % case["Wh"], n // case["Wh"]
                    pos = torch.stack([y // case["Hh"], y % case["Hh"], x], dim=-1)
                r[b] = _exact_turn(t[b].double(), pos, _split(case), case["pairing"], -1.0 if case["backward"] else 1.0)
            out.append(r)
        return out
    c = s["cache"]
    lens, counts, slots = _lengths(case), _counts(case), c["seq"][:, 1].tolist()
    table = c["page_table"].tolist()
    if case["op"] == "append":
        out = {x: c[x].double() for x in ("k_pages", "v_pages", "k_scale", "v_scale", "k_tail", "v_tail")}
        out["seq"] = None
        if B * case["H"] * (N // BLOCK + 2) > 20000:
            return None
        for b in range(B):
            L, n = lens[b], counts[b]
            if s["positions"] is not None:
                pos = s["positions"][b, :n]
            else:
                p = L + torch.arange(n, device="cuda")
                pos = torch.stack([p // (case["Hh"] * case["Wh"]), p // case["Wh"] % case["Hh"], p % case["Wh"]], dim=-1)
            kr = _exact_turn(s["k"][b, :, :n].double(), pos, _split(case), "adjacent", 1.0).to(torch.bfloat16).double()
            for name, new in (("k", kr), ("v", s["v"][b, :, :n].double())):
                old = c[name + "_tail"][b, slots[b], :, :L % BLOCK].double()
                rows = torch.cat([old, new], dim=1)
                first, last = L // BLOCK, (L + n) // BLOCK
                for j in range(first, last):
                    page = table[b][j]
                    for h in range(case["H"]):
                        codes, scale = _exact_codes(rows[h, (j - first) * BLOCK:(j - first + 1) * BLOCK])
                        out[name + "_pages"][page, h] = codes
                        out[name + "_scale"][page, h] = scale
                start = 0 if last > first else L % BLOCK
                slot = slots[b] if last == first else 1 - slots[b]
                end = (L + n) % BLOCK
                out[name + "_tail"][b, slot, :, start:end] = rows[:, (last - first) * BLOCK + start:(last - first) * BLOCK + end]
        return out
    Hq, H = case["Hq"], case["H"]
    o = torch.zeros(B, Hq, N, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, Hq, N, dtype=torch.float64, device="cuda")
    for b in range(B):
        L, n = lens[b], counts[b]
        if n == 0:
            continue
        p = L - n + torch.arange(n, device="cuda")
        if case["frame"]:
            group = torch.floor(p.double() / case["frame"]).long() * case["frame"]
            end = (group + case["frame"]).clamp(max=L)
        else:
            group, end = torch.full_like(p, L - n), torch.full_like(p, L)
        low = group - case["window"] if case["window"] >= 0 else torch.zeros_like(group)
        j = torch.arange(L, device="cuda")
        hidden = (j < low[:, None]) | (j >= end[:, None])
        pages = torch.tensor(table[b][:L // BLOCK], dtype=torch.long, device="cuda")
        for h in range(H):
            kv = []
            for name in ("k", "v"):
                x = c[name + "_pages"][pages, h].double() * c[name + "_scale"][pages, h].double()[:, None, None]
                kv.append(torch.cat([x.reshape(-1, d), c[name + "_tail"][b, slots[b], h, :L % BLOCK].double()]))
            for g in range(h * (Hq // H), (h + 1) * (Hq // H)):
                x = (s["q"][b, g, :n].double() @ kv[0].T) / math.sqrt(d)
                x[hidden] = -math.inf
                lse[b, g, :n] = torch.logsumexp(x, dim=-1) if L else -math.inf
                if L:
                    o[b, g, :n] = torch.nan_to_num(torch.softmax(x, dim=-1), nan=0.0) @ kv[1]
    return {"o": o, "lse": lse}
