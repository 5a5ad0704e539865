"""The 4-bit key/value cache with its attention, and the rotation ahead of it, as cases to measure.

A serving step: queries and keys of a fused q|k|v projection are normalised per head and
rotated by their positions, keys and values are quantised into 4-bit blocks, and each
sequence's last rows attend to everything it holds.  Kinds of case:

  rotate  norms (where there are weights) and rotation of the step's query and key heads
  write   append the step's rows, then read back every block that was touched
  attend  causal attention of the step's rows over the cache

A stored value is code * s * unit: codes -7 .. 7, one e4m3 scale s per token and 16 elements,
one unit for the keys and one for the values of a cache.  A block holds 16 tokens of a head:
8-byte atoms (16 codes plus 8, element e in nibble e) of the keys, those of the values, then
the scales of both in the atoms' order.

``own`` selects the framework's kernels; otherwise each pass is computed in
elementary torch operations in 32 bits (angles in 64).
"""
import math

import torch

own = False

K_UNIT, V_UNIT = 0.0537, 0.0291
EPS = 1e-6

_LARGEST_CODES = 32 * 32768 * 8 * 128       # codes of the keys a case may hold
_LARGEST_PAIRS = 32 * 8192 * 8192           # (query head, key) pairs of the largest score matrix
_LARGEST_PRODUCT = _LARGEST_PAIRS // 2 * 128  # pairs that are seen, times the head size
_LARGEST_ROWS = 16384 * 48 * 128            # elements of the rows a case rotates or writes


def listed():
    def case(name, kind, dtype="bf16", B=1, past=0, past_min=None, new=1, new_min=None, heads=(32, 8), D=128,
             page=64, window=0, holes=False, rotary=0, interleaved=False, base=10000.0, norm=False):
        return {"name": name, "kind": kind, "dtype": dtype, "B": B, "past": past,
                "past_min": past if past_min is None else past_min, "new": new,
                "new_min": new if new_min is None else new_min, "q_heads": heads[0], "kv_heads": heads[1], "D": D,
                "page": page, "window": window, "holes": holes, "rotary": rotary, "interleaved": interleaved,
                "base": base, "norm": norm}

    return [
        # one decode step of a small batch: launch latency
        case("rotate_decode_8", "rotate", B=8, past=700, past_min=3, rotary=128, norm=True),
        # far positions in 32 bits, part of a head rotated, pairs side by side
        case("rotate_f32_far", "rotate", dtype="f32", B=24, past=131071, past_min=1, new=333, new_min=1, heads=(10, 5),
             D=80, rotary=32, interleaved=True, holes=True),
        # prompts of unequal lengths
        case("rotate_prompts", "rotate", B=6, past=900, past_min=0, new=8192, new_min=777, rotary=128, base=500000.0,
             norm=True),
        # short sequences in 32 bits, heads of 80, blocks cut in the middle
        case("write_short_f32", "write", dtype="f32", B=3, past=5, past_min=0, new=333, new_min=1, heads=(10, 5), D=80,
             page=16),
        # one decode step of a full batch, every head with keys of its own (4096 = 32 x 128)
        case("write_decode_256", "write", B=256, past=5000, past_min=1, heads=(32, 32)),
        # prompts of unequal lengths, some of them continued in the middle of a block
        case("write_prompts", "write", B=6, past=900, past_min=0, new=8192, new_min=777),
        # one user, one token
        case("decode_1", "attend", B=1, past=776),
        # the decode step of a batch of 32 at hidden size 4096 (32 heads, each with its own keys)
        case("decode_32_mha", "attend", B=32, past=4096, past_min=129, heads=(32, 32), holes=True),
        # a large batch with long contexts
        case("decode_32_long", "attend", B=32, past=32767, past_min=32001),
        # drafted tokens checked in 32 bits under a window
        case("drafts_f32_window", "attend", dtype="f32", B=16, past=3000, past_min=0, new=5, new_min=1,
             heads=(12, 4), D=64, page=16, window=1024, holes=True),
        # prompts of unequal lengths after a shared prefix
        case("prompts_4", "attend", B=4, past=1024, past_min=0, new=2048, new_min=511),
        # one long prompt
        case("prompt_1_long", "attend", B=1, new=8192),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))

    kind = rng.choice(["rotate", "write", "attend", "attend"])
    c = {"kind": kind, "dtype": rng.choice(["bf16", "bf16", "bf16", "f32"]),
         "kv_heads": rng.choice([1, 2, 4, 5, 8, 8, 16, 32]), "D": rng.choice([64, 80, 96, 128, 128, 128, 256]),
         "page": rng.choice([16, 32, 64, 64, 128]), "holes": rng.random() < 0.3, "rotary": 0, "interleaved": False,
         "base": 10000.0, "norm": False}
    most_g = max(1, 64 // c["kv_heads"])
    c["q_heads"] = c["kv_heads"] * rng.choice([g for g in (1, 2, 3, 4, 6, 7, 8, 16) if g <= most_g])
    c["window"] = spread(16, 4096) if kind == "attend" and rng.random() < 0.2 else 0
    if kind == "rotate":
        c["rotary"] = rng.choice([c["D"], c["D"], c["D"] // 32 * 16])
        c["interleaved"] = rng.random() < 0.3
        c["base"] = rng.choice([10000.0, 500000.0, 1000000.0])
        c["norm"] = rng.random() < 0.6
    c["B"] = spread(1, 256)
    form = rng.choice(["tokens", "tokens", "few", "prompts"])
    c["new"] = 1 if form == "tokens" else rng.randint(2, 12) if form == "few" else spread(17, 8192)
    c["past"] = spread(1, 131072 if form == "tokens" else 8192)
    while True:   # within the largest listed cases
        total = c["past"] + c["new"]
        if (c["B"] * (total * c["kv_heads"] + 4 * c["new"] * c["q_heads"]) * c["D"] <= 0.98 * _LARGEST_CODES and
                (kind != "attend" or (
                    c["B"] * c["new"] * total * c["q_heads"] <= _LARGEST_PAIRS and
                    c["B"] * c["new"] * (c["past"] + c["new"] / 2) * c["q_heads"] * c["D"] <= _LARGEST_PRODUCT)) and
                (kind == "attend" or
                 c["B"] * c["new"] * (c["q_heads"] + 2 * c["kv_heads"]) * c["D"] <= _LARGEST_ROWS)):
            break
        if c["B"] > 1 and (rng.random() < 0.5 or total < 64):
            c["B"] = max(1, c["B"] // 2)
        else:
            c["past"] = max(1, c["past"] // 2)
            c["new"] = max(1, c["new"] // 2 + 1) if c["new"] > 1 else 1
    c["past_min"] = c["past"] if c["B"] == 1 or rng.random() < 0.3 else rng.randint(0, c["past"])
    c["new_min"] = c["new"] if c["new"] == 1 or rng.random() < 0.3 else rng.randint(1, c["new"])
    return c


def _step(case):
    """Rows and lengths (after the step) of each sequence: (new, length), spread over the case's ranges."""
    out = []
    for b in range(case["B"]):
        u, v = ((b + 1) * 0.6180339887498949) % 1.0, ((b + 1) * 0.7548776662466927) % 1.0
        n = case["new"] if b == 0 else case["new_min"] + int(u * (case["new"] - case["new_min"] + 1))
        p = case["past"] if b == 0 else case["past_min"] + int(v * (case["past"] - case["past_min"] + 1))
        length = p + n
        if case["holes"] and b % 5 == 3:     # a slot of the batch that holds nothing, or less than its rows
            length = 0 if b % 2 else n // 2
        out.append((n, length))
    return out


def _exclusive(values):
    out = [0]
    for v in values:
        out.append(out[-1] + v)
    return out


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    step = _step(case)
    B, Hq, H, D, ps = case["B"], case["q_heads"], case["kv_heads"], case["D"], case["page"]
    kind = case["kind"]
    rows = [n for n, _ in step]
    T = sum(rows)
    tdt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    s = {"kind": kind, "case": case, "max_new": max(rows),
         "lengths": torch.tensor([length for _, length in step], dtype=torch.int32, device=dev)}
    s["offsets"] = None if s["max_new"] == 1 else torch.tensor(_exclusive(rows), dtype=torch.int32, device=dev)
    # the step's rows, as the fused projection leaves them
    qkv = torch.empty((T, Hq + 2 * H, D), device=dev).normal_(generator=g)
    qkv[:, Hq:] *= torch.empty((T, 1, 1), device=dev).normal_(0.0, 0.4, generator=g).exp_()
    qkv = qkv.to(tdt)
    s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    if kind == "rotate":
        R = case["rotary"]
        s["freq"] = [case["base"] ** (-2.0 * i / R) for i in range(R // 2)]
        s["q_weight"] = s["k_weight"] = None
        if case["norm"]:
            s["q_weight"], s["k_weight"] = torch.empty((2, D), device=dev).normal_(1.0, 0.2, generator=g)
        s["q_out"] = torch.empty((T, Hq, D), dtype=tdt, device=dev)
        s["k_out"] = torch.empty((T, H, D), dtype=tdt, device=dev)
        if own:
            from heterogeneous_lora_gemm_gb300 import Rotary
            s["rotary"] = Rotary(D, freq=s["freq"], interleaved=case["interleaved"], device=s["q"].device)
        return s
    width = max(1, max(-(-length // ps) for _, length in step))
    used = [-(-length // ps) for _, length in step]
    n_pages = sum(used) + 3 + sum(used) // 8     # some pages belong to nobody; the last one is never in a table
    order = torch.randperm(n_pages - 1, generator=g, device=dev, dtype=torch.int32).cpu()
    pages = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b, u in enumerate(used):
        pages[b, :u] = order[at:at + u]
        at += u
    s["pages"] = pages.to(dev)
    # what the blocks hold: codes of normal values, scales of keys and values of unequal tokens; 255, a scale that
    # is no number, where nothing was written
    blocks = torch.empty((n_pages, H, ps // 16, 18 * D), dtype=torch.uint8, device=dev)
    some = max(1, (1 << 25) // (H * (ps // 16) * 18 * D))
    for i in range(0, n_pages, some):
        part = blocks[i:i + some]
        code = torch.randn(tuple(part.shape[:3]) + (16 * D, 2), generator=g, device=dev, dtype=torch.float16)
        code = code.mul_(3.2).round_().clamp_(-7, 7).add_(8).to(torch.uint8)
        part[..., :16 * D] = code[..., 0] | code[..., 1] << 4
        size = torch.empty(tuple(part.shape[:3]) + (2 * D,), device=dev).normal_(0.0, 0.4, generator=g).exp_()
        size[..., :D] *= 0.3 / K_UNIT
        size[..., D:] *= 0.2 / V_UNIT
        part[..., 16 * D:] = size.to(torch.float8_e4m3fn).view(torch.uint8)
    blocks[order[at:].to(dev).long()] = 255
    blocks[n_pages - 1] = 255
    k_at, v_at = (t.to(dev) for t in _atoms(D))
    for b, (n, length) in enumerate(step):
        held = length if kind == "attend" else max(0, length - n)
        if held < used[b] * ps:      # tokens that nothing has been written to
            page, first = pages[b, held // ps:used[b]].tolist(), held % ps
            where = torch.cat([16 * D + k_at[first % 16:].flatten(), 17 * D + v_at[first % 16:].flatten()])
            blocks[page[0], :, first // 16, where] = 255
            blocks[page[0], :, first // 16 + 1:] = 255
            blocks[torch.tensor(page[1:], dtype=torch.long, device=dev)] = 255
    s["blocks"] = blocks
    if kind == "attend":
        s["o"] = torch.empty((T, Hq, D), dtype=tdt, device=dev)
        s["scale"] = D ** -0.5
    else:                   # rows to read back: the blocks that the step touched
        back = [min(length, n + max(length - n, 0) % ps) for n, length in step]
        # (of them the tokens that the cache held are read too)
        s["back"] = torch.tensor(_exclusive(back), dtype=torch.int32, device=dev)
        s["max_back"] = max(1, max(back))
        s["k_back"] = torch.empty((sum(back), H, D), dtype=tdt, device=dev)
        s["v_back"] = torch.empty((sum(back), H, D), dtype=tdt, device=dev)
    if own:
        from heterogeneous_lora_gemm_gb300 import Cache4
        s["cache"] = Cache4(blocks, Hq, k_unit=K_UNIT, v_unit=V_UNIT)
    return s


def _atoms(D):
    """Index of the atom of token t, group n (16 elements) in a block: ([16, D / 16] of keys, of values)."""
    N = D // 16
    t, n = torch.arange(16)[:, None], torch.arange(N)[None, :]
    k = n // 4 * 64 + (t % 8 * (N - n // 4 * 4).clamp(max=4) + n % 4) * 2 + t // 8
    v = n // 8 * 128 + (t // 8 * (N - n // 8 * 8).clamp(max=8) + n % 8) * 8 + t % 8
    return k, v


def run(state):
    if own:
        return _run_own(state)
    if state["kind"] == "rotate":
        return [_plain_rotate(state, state[x], state[x + "_weight"]) for x in ("q", "k")]
    if state["kind"] == "attend":
        return _plain_attend(state)
    for x, first in (("k", True), ("v", False)):
        _plain_append(state, state[x], first)
    return [_plain_read(state, state["k_back"], True), _plain_read(state, state["v_back"], False)]


def _run_own(s):
    if s["kind"] == "rotate":
        s["rotary"].apply(s["q"], s["k"], s["lengths"], offsets=s["offsets"], max_new=s["max_new"],
                          q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, q_out=s["q_out"], k_out=s["k_out"])
        return [s["q_out"], s["k_out"]]
    c = s["cache"]
    if s["kind"] == "attend":
        c.attend(s["q"], s["o"], s["lengths"], s["pages"], offsets=s["offsets"], max_new=s["max_new"],
                 scale=s["scale"], window=s["case"]["window"])
        return s["o"]
    c.append(s["k"], s["v"], s["lengths"], s["pages"], offsets=s["offsets"], max_new=s["max_new"])
    c.read(s["k_back"], s["v_back"], s["lengths"], s["pages"], offsets=s["back"], max_new=s["max_back"])
    return [s["k_back"], s["v_back"]]


# ---- plain forms ---------------------------------------------------------- #
def _offsets(s, key="offsets"):
    if s[key] is not None:
        return s[key].long()
    return torch.arange(s["lengths"].numel() + 1, device=s["lengths"].device)


def _rows_of(s, offsets, T):
    """Sequence and position of each row."""
    r = torch.arange(T, device=offsets.device)
    b = torch.searchsorted(offsets, r, right=True) - 1
    return b, s["lengths"].long()[b] - offsets[b + 1] + r


def _plain_rotate(s, x, weight):
    case = s["case"]
    R, T = case["rotary"], x.shape[0]
    _, pos = _rows_of(s, _offsets(s), T)
    freq = torch.tensor(s["freq"], dtype=torch.float64, device=x.device)
    angle = pos.double()[:, None] * freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt((y * y).mean(dim=-1, keepdim=True) + EPS) * weight
    if case["interleaved"]:
        a, b = y[..., 0:R:2], y[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    else:
        a, b = y[..., :R // 2], y[..., R // 2:R]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    y = torch.cat([turned, y[..., R:]], dim=-1)
    return torch.where((pos >= 0)[:, None, None], y, torch.zeros_like(y)).to(x.dtype)


def _plain_values(blocks, keys):
    """Blocks [..., 18 D] as values in 32 bits [..., 16, D]; tokens that were never written may be no numbers."""
    D = blocks.shape[-1] // 18
    at = _atoms(D)[0 if keys else 1].to(blocks.device)
    first, scales = (0, 16 * D) if keys else (8 * D, 17 * D)
    atoms = blocks[..., first:first + 8 * D].unflatten(-1, (D, 8))[..., at, :]
    code = torch.stack([atoms & 15, atoms >> 4], dim=-1).flatten(-2).float() - 8.0
    scale = blocks[..., scales:scales + D][..., at].contiguous().view(torch.float8_e4m3fn).float()
    return (code * scale[..., None] * (K_UNIT if keys else V_UNIT)).flatten(-2)


def _plain_read(s, like, keys):
    ps = s["case"]["page"]
    offsets, blocks = _offsets(s, "back"), s["blocks"]
    b, pos = _rows_of(s, offsets, like.shape[0])
    at = pos.clamp(min=0)
    page = s["pages"].long()[b, (at // ps).clamp(max=s["pages"].shape[1] - 1)].clamp(min=0)
    D = like.shape[2]
    atom = _atoms(D)[0 if keys else 1].to(like.device)[at % 16]                         # [rows, groups]
    held = blocks[page, :, at % ps // 16]                                              # [rows, heads, 18 D]
    first, scales = (0, 16 * D) if keys else (8 * D, 17 * D)
    wide = (like.shape[0], like.shape[1], D // 16)
    index = (atom[:, None, :, None] * 8 + torch.arange(8, device=like.device)).expand(wide + (8,)).flatten(2)
    codes = held.gather(2, first + index).unflatten(2, (D // 16, 8))
    code = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).float() - 8.0
    scale = held.gather(2, (scales + atom[:, None]).expand(wide)).view(torch.float8_e4m3fn).float()
    x = (code * scale[..., None] * (K_UNIT if keys else V_UNIT)).flatten(-2)
    return torch.where((pos >= 0)[:, None, None], x, torch.zeros_like(x)).to(like.dtype)


def _plain_append(s, rows, keys):
    ps, blocks = s["case"]["page"], s["blocks"]
    offsets, (T, H, D) = _offsets(s), rows.shape
    unit = torch.tensor(K_UNIT if keys else V_UNIT, device=rows.device)
    b, pos = _rows_of(s, offsets, T)
    x = rows.float().unflatten(2, (D // 16, 16))
    top = x.abs().amax(dim=-1)
    one = torch.ones_like(top)
    scale = (top * (one / (7.0 * unit))).clamp(max=448.0).to(torch.float8_e4m3fn)
    step = scale.float() * unit
    inv = torch.where(step > 0, one / step, torch.zeros_like(step))
    code = (torch.round(x * inv[..., None]).clamp(-7, 7) + 8.0).to(torch.uint8)
    atoms = code[..., 0::2] | code[..., 1::2] << 4                                     # [T, H, groups, 8]
    seen = (pos >= 0).nonzero().flatten()
    b, pos = b[seen], pos[seen]
    page = s["pages"].long()[b, pos // ps]
    atom = _atoms(D)[0 if keys else 1].to(rows.device)[pos % 16]
    first, scales = (0, 16 * D) if keys else (8 * D, 17 * D)
    heads = torch.arange(H, device=rows.device)
    to = (page[:, None] * H + heads) * (ps // 16) + (pos % ps // 16)[:, None]          # block of each row and head
    flat = blocks.view(-1)
    at = to[:, :, None] * (18 * D) + atom[:, None]
    flat[at + scales] = scale[seen].view(torch.uint8)
    at = to[:, :, None, None] * (18 * D) + first + atom[:, None, :, None] * 8 + torch.arange(8, device=rows.device)
    flat[at] = atoms[seen]


def _plain_attend(s):
    ps = s["case"]["page"]
    B, width = s["pages"].shape
    blocks, dev = s["blocks"], s["blocks"].device
    H, D = s["case"]["kv_heads"], s["case"]["D"]
    L = width * ps
    offsets, length = _offsets(s), s["lengths"].long()
    n = offsets[1:] - offsets[:-1]
    N, T, Hq = s["max_new"], s["q"].shape[0], s["q"].shape[1]
    page = s["pages"].long().clamp(min=0)
    held = (torch.arange(L, device=dev) < length[:, None]).view(B, 1, L, 1)

    def restored(keys):
        x = torch.empty((B, H, L, D), device=dev)
        for b in range(B):
            x[b] = _plain_values(blocks[page[b]], keys).permute(1, 0, 2, 3, 4).reshape(H, L, D)
        return x.masked_fill_(~held, 0.0)

    i = torch.arange(N, device=dev)
    q = s["q"][(offsets[:-1, None] + i).clamp(max=T - 1)].float()
    q = q.view(B, N, H, Hq // H, D).permute(0, 2, 1, 3, 4).reshape(B, H, -1, D)
    x = torch.matmul(q, restored(True).transpose(2, 3)).mul_(s["scale"]).view(B, H, N, Hq // H, L)
    pos = (length - n)[:, None] + i
    t = torch.arange(L, device=dev)
    seen = t <= pos[:, :, None]
    if s["case"]["window"]:
        seen &= t > pos[:, :, None] - s["case"]["window"]
    x.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = x.amax(dim=-1, keepdim=True)
    x.sub_(torch.where(torch.isfinite(m), m, torch.zeros_like(m))).exp_()
    total = x.sum(dim=-1, keepdim=True)
    o = torch.matmul(x.view(B, H, -1, L), restored(False)).view(B, H, N, Hq // H, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    b, at = _rows_of(s, offsets, T)
    return o[b, :, at - (length - n)[b]].reshape(T, Hq, D).to(s["q"].dtype)


# ---- what a pass cannot do without ---------------------------------------- #
def work(case):
    H, Hq, D, e = case["kv_heads"], case["q_heads"], case["D"], 2 if case["dtype"] == "bf16" else 4
    step = _step(case)
    if case["kind"] == "rotate":
        n = sum(n for n, _ in step) * (Hq + H) * D
        return {"bytes": 2 * n * e, "flops": n * (4 if case["norm"] else 0) + n // D * case["rotary"] * 3}
    if case["kind"] == "write":
        new = sum(min(n, length) for n, length in step) * H * D
        back = sum(min(length, n + max(length - n, 0) % case["page"]) for n, length in step) * H * D
        return {"bytes": 2 * (new * e + new * 9 // 16 + back * 9 // 16 + back * e), "flops": 2 * (3 * new + back)}
    codes = pairs = 0
    for n, length in step:
        w = case["window"] or length
        lo = max(0, length - n - w + 1)
        codes += max(0, length - lo) * H * D
        full = max(0, length - n)                      # position of the first row that sees anything
        if length:
            k = length - full                          # rows at positions full .. length - 1
            short = min(max(0, min(w, length) - full), k)   # of them, those that see fewer than w tokens
            pairs += short * full + short * (short + 1) // 2 + (k - short) * w
    return {"bytes": 2 * codes * 9 // 16 + 2 * sum(n for n, _ in step) * Hq * D * e, "flops": 4 * D * pairs * Hq}


# ---- from the definitions, in 64 bits ------------------------------------- #
def exact(case, seed):
    s = prepare(case, seed)
    step = _step(case)
    rows = _exclusive([n for n, _ in step])
    if case["kind"] == "rotate":
        return [_exact_rotate(s, step, rows, x) for x in ("q", "k")]
    if case["kind"] == "attend":
        return _exact_attend(s, step, rows)
    return [_exact_write(s, step, rows, x) for x in ("k", "v")]


def _exact_rotate(s, step, rows, which):
    case, x = s["case"], s[which].double()
    R, w = case["rotary"], s[which + "_weight"]
    if w is not None:
        x = x * w.double() / (x.square().mean(-1, keepdim=True) + EPS).sqrt()
    freq = torch.tensor(s["freq"], dtype=torch.float64, device="cuda")
    order = torch.arange(R).view(-1, 2) if case["interleaved"] else torch.arange(R).view(2, -1).T
    out = x.clone()
    for b, (n, length) in enumerate(step):
        at = slice(rows[b], rows[b + 1])
        pos = torch.arange(length - n, length, dtype=torch.float64, device="cuda")
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos[:, None, None] * freq)
        z = torch.complex(x[at][..., order[:, 0]], x[at][..., order[:, 1]]) * turn
        out[at, :, order[:, 0]] = z.real
        out[at, :, order[:, 1]] = z.imag
        out[at] *= (pos >= 0).double()[:, None, None]
    return out


def _exact_token(block, t, keys):
    """Values of token t of blocks [H, 18 D]: atom by atom."""
    D = block.shape[-1] // 18
    at = _atoms(D)[0 if keys else 1][t].tolist()
    first, scales = (0, 16 * D) if keys else (8 * D, 17 * D)
    parts = []
    for a in at:
        codes = block[:, first + 8 * a:first + 8 * a + 8].int()
        code = torch.stack([codes % 16, codes // 16], dim=-1).view(-1, 16).double() - 8
        byte = block[:, scales + a].double()
        e, m = (byte % 128 / 8).floor(), byte % 8
        size = torch.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7), m * 2.0 ** -9)
        size = torch.where(byte % 128 == 127, torch.full_like(size, math.nan), size)
        parts.append(code * (size * float(torch.tensor(K_UNIT if keys else V_UNIT)))[:, None])
    return torch.cat(parts, dim=-1)


def _exact_held(s, b, length, keys):
    """Values [H, length, D] that sequence b holds."""
    blocks, D = s["blocks"], s["case"]["D"]
    held = s["pages"][b, :-(-length // s["case"]["page"])].long()
    of = blocks[held].transpose(0, 1).flatten(1, 2)                  # [H, blocks, 18 D]
    tokens = [_exact_token(of.reshape(-1, 18 * D), t, keys).view(of.shape[0], -1, D) for t in range(16)]
    return torch.stack(tokens, dim=2).flatten(1, 2)[:, :length]


def _exact_write(s, step, rows, which):
    case, keys = s["case"], which == "k"
    unit, H, D = float(torch.tensor(K_UNIT if keys else V_UNIT)), case["kv_heads"], case["D"]
    out = []
    for b, (n, length) in enumerate(step):
        if not length:
            continue
        back, start = min(length, n + max(length - n, 0) % case["page"]), max(0, length - n)
        new = s[which][rows[b + 1] - (length - start):rows[b + 1]].double().view(-1, H, D // 16, 16)
        size = new.abs().amax(-1) / 7 / unit
        grid = 2.0 ** (torch.frexp(size.clamp(min=2.0 ** -6))[1].double() - 4)      # steps of e4m3 at that size
        size = (torch.round(size / grid) * grid).clamp(max=448)
        step_of = (size * unit)[..., None].clamp(min=1e-300)
        new = (torch.round(new / step_of).clamp(-7, 7) * (size * unit)[..., None]).view(-1, H, D)
        old = _exact_held(s, b, start, keys).transpose(0, 1) if start else new[:0]
        out.append(torch.cat([old, new])[length - back:])
    return torch.cat(out)


def _exact_attend(s, step, rows):
    case, H = s["case"], s["case"]["kv_heads"]
    G = case["q_heads"] // H
    out = torch.zeros(s["o"].shape, dtype=torch.float64, device="cuda")
    for b, (n, length) in enumerate(step):
        if not length:
            continue
        keys, values = _exact_held(s, b, length, True), _exact_held(s, b, length, False)
        pos = torch.arange(length - n, length, device="cuda")[:, None]
        t = torch.arange(length, device="cuda")
        hidden = t > pos
        if case["window"]:
            hidden |= t <= pos - case["window"]
        for h in range(H):
            for g in range(h * G, h * G + G):
                w = (s["q"][rows[b]:rows[b + 1], g].double() @ keys[h].T) * s["scale"]
                w = w.masked_fill_(hidden, -math.inf).softmax(dim=-1)
                w = torch.where(pos >= 0, w, torch.zeros_like(w))
                out[rows[b]:rows[b + 1], g] = w @ values[h]
    return out
