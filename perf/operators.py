"""The 8-bit key/value cache and its attention, as cases to measure.

A serving step of a paged cache: rows of a fused q|k|v projection come in, keys and
values are quantised into int8 pages (one fp32 scale per page and head), and each
sequence's last rows attend to everything it holds.  Kinds of case:

  write   append the step's rows, then read back every block that was touched
  read    restore whole sequences into rows
  attend  causal attention of the step's rows over the cache

``own`` selects the framework's kernels; otherwise each pass is computed in
elementary torch operations in 32 bits.
"""
import math

import torch

own = False

_LARGEST_CODES = 32 * 32768 * 8 * 128       # codes of the keys a case may hold
_LARGEST_PAIRS = 32 * 8192 * 8192           # (query head, key) pairs of the largest score matrix
_LARGEST_PRODUCT = _LARGEST_PAIRS // 2 * 128  # pairs that are seen, times the head size


def listed():
    def case(name, kind, dtype="bf16", B=1, past=0, past_min=None, new=1, new_min=None, heads=(32, 8), D=128,
             page=64, window=0, holes=False):
        return {"name": name, "kind": kind, "dtype": dtype, "B": B, "past": past,
                "past_min": past if past_min is None else past_min, "new": new,
                "new_min": new if new_min is None else new_min, "q_heads": heads[0], "kv_heads": heads[1], "D": D,
                "page": page, "window": window, "holes": holes}

    return [
        # one decode step of a small batch: launch latency
        case("write_decode_8", "write", B=8, past=700, past_min=3, page=16, holes=True),
        # one decode step of a full batch, every head with keys of its own (4096 = 32 x 128)
        case("write_decode_256", "write", B=256, past=5000, past_min=1, heads=(32, 32)),
        # prompts of unequal lengths, some of them continued in the middle of a block
        case("write_prompts", "write", B=6, past=900, past_min=0, new=8192, new_min=777),
        # short sequences leave the cache in 32 bits, heads of 80
        case("read_short_f32", "read", dtype="f32", B=3, past=5, past_min=0, new=333, new_min=1, heads=(10, 5), D=80,
             page=16),
        # whole sequences leave the cache (moved to another server)
        case("read_long", "read", B=8, new=16384, new_min=9001),
        # one user, one token
        case("decode_1", "attend", B=1, past=776),
        # the decode step of a batch of 32 at hidden size 4096 (32 heads, each with its own keys)
        case("decode_32_mha", "attend", B=32, past=4096, past_min=129, heads=(32, 32), holes=True),
        # few users with very long contexts
        case("decode_4_long", "attend", B=4, past=131071, past_min=90000, heads=(64, 8), page=128),
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

    kind = rng.choice(["write", "read", "attend", "attend", "attend", "attend"])
    c = {"kind": kind, "dtype": rng.choice(["bf16", "bf16", "bf16", "f32"]),
         "kv_heads": rng.choice([1, 2, 4, 5, 8, 8, 16, 32]), "D": rng.choice([64, 80, 96, 128, 128, 128, 256]),
         "page": rng.choice([16, 32, 64, 64, 128]), "holes": rng.random() < 0.3}
    most_g = max(1, 64 // c["kv_heads"])
    c["q_heads"] = c["kv_heads"] * rng.choice([g for g in (1, 2, 3, 4, 6, 7, 8, 16) if g <= most_g])
    c["window"] = spread(16, 4096) if kind == "attend" and rng.random() < 0.2 else 0
    c["B"] = spread(1, 256)
    form = rng.choice(["tokens", "tokens", "few", "prompts"]) if kind != "read" else "prompts"
    c["new"] = 1 if form == "tokens" else rng.randint(2, 12) if form == "few" else spread(17, 8192)
    c["past"] = spread(1, 131072 if form == "tokens" else 8192)
    while True:   # within the largest listed cases
        total = c["past"] + c["new"]
        if (c["B"] * (total * c["kv_heads"] + 4 * c["new"] * c["q_heads"]) * c["D"] <= 0.98 * _LARGEST_CODES and
                (kind != "attend" or (
                    c["B"] * c["new"] * total * c["q_heads"] <= _LARGEST_PAIRS and
                    c["B"] * c["new"] * (c["past"] + c["new"] / 2) * c["q_heads"] * c["D"] <= _LARGEST_PRODUCT)) and
                (kind == "attend" or c["B"] * c["new"] * c["kv_heads"] * c["D"] <= _LARGEST_CODES // 16)):
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
    width = max(1, max(-(-length // ps) for _, length in step))
    used = [-(-length // ps) for _, length in step]
    n_pages = sum(used) + 3 + sum(used) // 8     # some pages belong to nobody; the last one is never in a table
    order = torch.randperm(n_pages - 1, generator=g, device=dev, dtype=torch.int32).cpu()
    pages = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b, u in enumerate(used):
        pages[b, :u] = order[at:at + u]
        at += u
    s = {"kind": kind, "case": case}

    def codes():
        t = torch.randn((n_pages, H, ps, D), generator=g, device=dev, dtype=torch.float16)
        return t.mul_(32).round_().clamp_(-127, 127).to(torch.int8)

    def scales(size):
        t = torch.empty((n_pages, H), device=dev).normal_(0.0, 0.4, generator=g).exp_().mul_(size / 32)
        t[order[at:].to(dev).long()] = float("nan")      # what nobody owns
        t[n_pages - 1] = float("nan")
        return t

    s["k_codes"], s["v_codes"] = codes(), codes()
    s["k_scale"], s["v_scale"] = scales(1.5), scales(0.7)
    s["pages"] = pages.to(dev)
    s["lengths"] = torch.tensor([length for _, length in step], dtype=torch.int32, device=dev)
    tdt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    rows = [n for n, _ in step]
    T = sum(rows)
    s["max_new"] = max(rows)
    s["offsets"] = None if s["max_new"] == 1 else torch.tensor(_exclusive(rows), dtype=torch.int32, device=dev)
    if kind != "read":      # the step's rows, as the fused projection leaves them
        qkv = torch.empty((T, Hq + 2 * H, D), device=dev).normal_(generator=g)
        qkv[:, Hq:] *= torch.empty((T, 1, 1), device=dev).normal_(0.0, 0.4, generator=g).exp_()
        qkv = qkv.to(tdt)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    if kind == "attend":
        s["o"] = torch.empty((T, Hq, D), dtype=tdt, device=dev)
        s["scale"] = D ** -0.5
    else:                   # rows to read back: the blocks that the step touched, or what was asked for
        back = [n if kind == "read" else min(length, n + max(length - n, 0) % ps) for n, length in step]
        s["back"] = torch.tensor(_exclusive(back), dtype=torch.int32, device=dev)
        s["max_back"] = max(1, max(back))
        s["k_back"] = torch.empty((sum(back), H, D), dtype=tdt, device=dev)
        s["v_back"] = torch.empty((sum(back), H, D), dtype=tdt, device=dev)
    if own:
        from heterogeneous_lora_gemm_gb300 import Cache
        s["cache"] = Cache(s["k_codes"], s["k_scale"], s["v_codes"], s["v_scale"], Hq)
    return s


def run(state):
    if own:
        return _run_own(state)
    if state["kind"] == "attend":
        return _plain_attend(state)
    if state["kind"] == "write":
        for x in ("k", "v"):
            _plain_append(state, state[x], state[x + "_codes"], state[x + "_scale"])
    k, v = (_plain_read(state, state[x + "_codes"], state[x + "_scale"], state[x + "_back"]) for x in ("k", "v"))
    return _stored(state, k, v)


def _stored(s, k, v):
    """What a write leaves: the restored blocks and the scales (those of the last page mean nothing)."""
    return [k, v] if s["kind"] == "read" else [k, v, s["k_scale"][:-1], s["v_scale"][:-1]]


def _run_own(s):
    c = s["cache"]
    if s["kind"] == "attend":
        c.attend(s["q"], s["o"], s["lengths"], s["pages"], offsets=s["offsets"], max_new=s["max_new"],
                 scale=s["scale"], window=s["case"]["window"])
        return s["o"]
    if s["kind"] == "write":
        c.append(s["k"], s["v"], s["lengths"], s["pages"], offsets=s["offsets"], max_new=s["max_new"])
    c.read(s["k_back"], s["v_back"], s["lengths"], s["pages"], offsets=s["back"], max_new=s["max_back"])
    return _stored(s, s["k_back"], s["v_back"])


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


def _plain_read(s, codes, scale, like):
    offsets, ps = _offsets(s, "back"), codes.shape[2]
    b, pos = _rows_of(s, offsets, like.shape[0])
    seen = pos >= 0
    at = pos.clamp(min=0)
    page = s["pages"].long()[b, (at // ps).clamp(max=s["pages"].shape[1] - 1)].clamp(min=0)
    x = codes[page, :, at % ps].float() * scale[page][:, :, None]
    return torch.where(seen[:, None, None], x, torch.zeros_like(x)).to(like.dtype)


def _plain_append(s, rows, codes, scale):
    offsets, ps = _offsets(s), codes.shape[2]
    B, width = s["pages"].shape
    H, D, dev = codes.shape[1], codes.shape[3], codes.device
    length = s["lengths"].long()
    start = (length - (offsets[1:] - offsets[:-1])).clamp(min=0)      # tokens held before the step
    first = start // ps
    blocks = (s["max_new"] - 1) // ps + 2
    j = first[:, None] + torch.arange(blocks, device=dev)
    touched = (j * ps < length[:, None]) & (length > start)[:, None]
    page = s["pages"].long()[torch.arange(B, device=dev)[:, None], j.clamp(max=width - 1)].clamp(min=0)
    page = torch.where(touched, page, torch.full_like(page, codes.shape[0] - 1))
    b, pos = _rows_of(s, offsets, rows.shape[0])
    slot = torch.where(pos >= 0, pos - first[b] * ps, torch.full_like(pos, blocks * ps))
    new = torch.zeros((B, blocks * ps + 1, H, D), device=dev)
    new[b, slot] = rows.float()
    new = new[:, :-1].view(B, blocks, ps, H, D).permute(0, 1, 3, 2, 4)   # as a page lies: [head, token, D]
    at = j[:, :, None] * ps + torch.arange(ps, device=dev)              # position of each token of a block
    is_old = (at < start[:, None, None])[:, :, None, :, None]
    is_new = ((at >= start[:, None, None]) & (at < length[:, None, None]))[:, :, None, :, None]
    top = torch.where(is_new, new.abs(), torch.zeros_like(new)).amax(dim=(3, 4))
    held = (j * ps < start[:, None])[:, :, None]
    s_old = torch.where(held, scale[page], torch.zeros_like(top))
    s_new = torch.maximum(s_old, top / torch.full_like(top, 127.0))
    inv = torch.where(s_new >= 2.0 ** -120, torch.ones_like(s_new) / s_new, torch.zeros_like(s_new))
    was = codes[page]
    x = torch.where(is_old, was.float() * s_old[..., None, None], new)
    c = torch.round(x * inv[..., None, None]).clamp(-127, 127)
    codes[page] = torch.where(is_old | is_new, c, was.float()).to(torch.int8)
    scale[page] = s_new


def _plain_attend(s):
    codes, ps = s["k_codes"], s["case"]["page"]
    B, width = s["pages"].shape
    H, D, dev = codes.shape[1], codes.shape[3], codes.device
    L = width * ps
    offsets, length = _offsets(s), s["lengths"].long()
    n = offsets[1:] - offsets[:-1]
    N, T, Hq = s["max_new"], s["q"].shape[0], s["q"].shape[1]
    page = s["pages"].long().clamp(min=0)
    held = (torch.arange(L, device=dev) < length[:, None]).view(B, width, 1, ps, 1)

    def restored(codes, scale):
        x = codes[page].float().mul_(scale[page][..., None, None])
        return x.masked_fill_(~held, 0.0).permute(0, 2, 1, 3, 4).reshape(B, H, L, D)

    i = torch.arange(N, device=dev)
    q = s["q"][(offsets[:-1, None] + i).clamp(max=T - 1)].float()
    q = q.view(B, N, H, Hq // H, D).permute(0, 2, 1, 3, 4).reshape(B, H, -1, D)
    x = torch.matmul(q, restored(codes, s["k_scale"]).transpose(2, 3)).mul_(s["scale"]).view(B, H, N, Hq // H, L)
    pos = (length - n)[:, None] + i
    t = torch.arange(L, device=dev)
    seen = t <= pos[:, :, None]
    if s["case"]["window"]:
        seen &= t > pos[:, :, None] - s["case"]["window"]
    x.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = x.amax(dim=-1, keepdim=True)
    x.sub_(torch.where(torch.isfinite(m), m, torch.zeros_like(m))).exp_()
    total = x.sum(dim=-1, keepdim=True)
    o = torch.matmul(x.view(B, H, -1, L), restored(s["v_codes"], s["v_scale"])).view(B, H, N, Hq // H, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    b, at = _rows_of(s, offsets, T)
    return o[b, :, at - (length - n)[b]].reshape(T, Hq, D).to(s["q"].dtype)


# ---- what a pass cannot do without ---------------------------------------- #
def work(case):
    H, Hq, D, e = case["kv_heads"], case["q_heads"], case["D"], 2 if case["dtype"] == "bf16" else 4
    step = _step(case)
    if case["kind"] == "read":
        codes = sum(min(n, length) for n, length in step) * H * D
        return {"bytes": 2 * codes + 2 * sum(n for n, _ in step) * H * D * e, "flops": 2 * codes}
    if case["kind"] == "write":
        new = sum(min(n, length) for n, length in step) * H * D
        back = sum(min(length, n + max(length - n, 0) % case["page"]) for n, length in step) * H * D
        return {"bytes": 2 * (new * e + new + back + back * e), "flops": 2 * (3 * new + back)}
    codes = pairs = 0
    for n, length in step:
        w = case["window"] or length
        lo = max(0, length - n - w + 1)
        codes += max(0, length - lo) * H * D
        full = max(0, length - n)                      # position of the first row that sees anything
        if length:
            k = length - full                          # rows at positions full .. length - 1
            short = max(0, min(w, length) - full)      # of them, those that see fewer than w tokens
            short = min(short, k)
            pairs += short * full + short * (short + 1) // 2 + (k - short) * w
    return {"bytes": 2 * codes + 2 * sum(n for n, _ in step) * Hq * D * e, "flops": 4 * D * pairs * Hq}


# ---- from the definitions, in 64 bits ------------------------------------- #
def exact(case, seed):
    s = prepare(case, seed)
    step, ps = _step(case), case["page"]
    rows = _exclusive([n for n, _ in step])
    table = s["pages"].cpu()
    if case["kind"] == "attend":
        return _exact_attend(s, step, rows, table)
    out = []
    for x in ("k", "v"):
        codes, scale = s[x + "_codes"].double(), s[x + "_scale"].double()
        if case["kind"] == "write":
            for b, (n, length) in enumerate(step):
                start = max(0, length - n)
                for j in range(start // ps, -(-length // ps)):
                    lo, hi, page = max(start - j * ps, 0), min(length - j * ps, ps), int(table[b, j])
                    r = rows[b] + n - length + j * ps + lo
                    new = s[x][r:r + hi - lo].double().transpose(0, 1)
                    held = scale[page] if lo > 0 else torch.zeros_like(scale[page])
                    old = codes[page, :, :lo] * held[:, None, None]
                    scale[page] = torch.maximum(held, new.abs().amax(dim=(1, 2)) / 127)
                    value = torch.cat([old, new], dim=1) / scale[page][:, None, None].clamp(min=1e-300)
                    codes[page, :, :hi] = torch.round(value).clamp(-127, 127)
        parts = []
        for b, (n, length) in enumerate(step):
            if case["kind"] == "write":
                n = min(length, n + max(length - n, 0) % ps)
            held = table[b, :-(-length // ps)].long().to(codes.device)
            y = (codes[held] * scale[held][:, :, None, None]).transpose(1, 2).reshape(-1, codes.shape[1], codes.shape[3])
            pad = torch.zeros((max(0, n - length),) + tuple(y.shape[1:]), dtype=y.dtype, device=y.device)
            parts.append(torch.cat([pad, y[max(0, length - n):length]]))
        out.append((torch.cat(parts), scale[:-1]))
    (k, ks), (v, vs) = out
    return [k, v] if case["kind"] == "read" else [k, v, ks, vs]


def _exact_attend(s, step, rows, table):
    case, H = s["case"], s["case"]["kv_heads"]
    G = case["q_heads"] // H
    out = torch.zeros(s["o"].shape, dtype=torch.float64, device="cuda")
    for b, (n, length) in enumerate(step):
        if not length:
            continue
        held = table[b, :-(-length // case["page"])].long().cuda()
        pos = torch.arange(length - n, length, device="cuda")[:, None]
        t = torch.arange(length, device="cuda")
        hidden = t > pos
        if case["window"]:
            hidden |= t <= pos - case["window"]
        for h in range(H):
            k, v = ((s[x + "_codes"][held, h].double() * s[x + "_scale"][held, h].double()[:, None, None])
                    .reshape(-1, case["D"])[:length] for x in ("k", "v"))
            for g in range(h * G, h * G + G):
                w = (s["q"][rows[b]:rows[b + 1], g].double() @ k.T) * s["scale"]
                w = w.masked_fill_(hidden, -math.inf).softmax(dim=-1)
                w = torch.where(pos >= 0, w, torch.zeros_like(w))
                out[rows[b]:rows[b + 1], g] = w @ v
    return out
