"""The 8-bit key/value cache and its attention through the public entry points, against
plain implementations: codes and scales bit for bit (the definition's fp32 operations in
numpy), attention in 64 bits.

Tolerance of an attention output o = sum p v, with A = sum p |v| and S the largest
scale * sum |q||k| of the row: the weights round to 8 bits at the least (2^-8 of A), a
score's fp32 sum of up to 256 terms is off by at most 2^-16 S (both into A), the output
rounds once.  bf16: 2^-8 |o| + (2^-7 + 2^-15 (1 + S)) A;  fp32: 2^-16 (1 + S) A.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():   # pragma: no cover - CPU machine
    pytest.skip("needs a GPU", allow_module_level=True)

from heterogeneous_lora_gemm_gb300 import Cache, mlora  # noqa: E402

TDT = {"bf16": torch.bfloat16, "f32": torch.float32}
F = np.float32


class Setup:
    """Pages with random contents, shuffled page tables, and NaN scales on pages nobody owns."""

    def __init__(self, lengths, H, D, ps, Hq=None, seed=0, spare=3, k_size=1.5, v_size=0.7):
        rng = np.random.default_rng(seed)
        self.lengths, self.H, self.D, self.ps, self.Hq = list(lengths), H, D, ps, Hq or H
        used = [-(-max(n, 0) // ps) for n in lengths]
        self.n_pages = sum(used) + spare
        order = rng.permutation(self.n_pages)
        self.width = max([1] + used)
        self.table = np.full((len(lengths), self.width), -7, np.int32)   # unused entries are never read
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = order[at:at + u]
            at += u
        shape = (self.n_pages, H, ps, D)
        self.kc, self.vc = (rng.integers(-127, 128, shape).astype(np.int8) for _ in range(2))
        self.ks, self.vs = ((rng.uniform(0.5, 2.0, shape[:2]) * z / 64).astype(F) for z in (k_size, v_size))
        self.ks[order[at:]] = self.vs[order[at:]] = np.nan
        self.upload()

    def upload(self):
        self.dev = [torch.from_numpy(x).cuda() for x in (self.kc, self.ks, self.vc, self.vs)]
        self.pages = torch.from_numpy(self.table).cuda()
        self.len = torch.tensor(self.lengths, dtype=torch.int32, device="cuda")
        self.cache = Cache(*self.dev, self.Hq)

    def values(self, codes, scale, b, dtype=np.float64):
        """[length, H, D] that sequence b holds."""
        n = self.lengths[b]
        t = self.table[b, :-(-n // self.ps)]
        x = codes[t].astype(dtype) * scale[t].astype(dtype)[:, :, None, None]
        return x.transpose(0, 2, 1, 3).reshape(-1, self.H, self.D)[:n]


def offsets_of(rows):
    return torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device="cuda")


def as_np(t):
    return t.detach().float().cpu().numpy()


# ---- append ---------------------------------------------------------------- #
def plain_append(codes, scale, x, table, lengths, rows, ps):
    """The definition, in fp32: codes and scales after the step."""
    codes, scale = codes.copy(), scale.copy()
    at = 0
    for b, (n, length) in enumerate(zip(rows, lengths)):
        start = length - n
        for j in range(max(start, 0) // ps, -(-length // ps)):
            lo, hi = max(start - j * ps, 0), min(length - j * ps, ps)
            if hi <= lo:
                continue
            page = table[b, j]
            new = x[at + j * ps + lo - start:at + j * ps + hi - start]           # [rows, H, D]
            for h in range(codes.shape[1]):
                held = scale[page, h] if lo > 0 else F(0)
                v = new[:, h].astype(F)
                finite = np.abs(np.where(np.isfinite(v), v, F(0)))
                s = max(held, finite.max() / F(127))
                with np.errstate(all="ignore"):
                    inv = F(1) / s if s >= F(2.0 ** -120) else F(0)
                    old = codes[page, h, :lo].astype(F) * held
                    q = np.concatenate([old, v]) * inv
                q = np.where(np.isnan(q), F(0), np.clip(q, F(-127), F(127)))
                codes[page, h, :hi] = np.rint(q).astype(np.int8)
                scale[page, h] = s
        at += n
    return codes, scale


def strided(x, dtype, pad_heads=0, transpose=False):
    """[T, H, D] on the GPU as a slice of wider rows, or stored heads first."""
    t = torch.from_numpy(x).to(TDT[dtype]).cuda()
    if transpose:
        return t.transpose(0, 1).contiguous().transpose(0, 1)
    if pad_heads:
        wide = torch.full((t.shape[0], t.shape[1] + pad_heads, t.shape[2]), float("nan"), dtype=t.dtype, device="cuda")
        wide[:, 1:1 + t.shape[1]] = t
        return wide[:, 1:1 + t.shape[1]]
    return t


APPENDS = [
    # rows, lengths after, H, D, page, dtype
    ([1, 1, 1, 1], [1, 17, 16, 33], 2, 64, 16, "bf16"),
    ([1], [1], 1, 16, 16, "f32"),
    ([5, 0, 40, 1], [5, 9, 100, 64], 3, 80, 32, "bf16"),
    ([70, 33], [70, 200], 2, 128, 64, "f32"),
    ([7, 3, 2], [3, 0, 2], 2, 128, 16, "bf16"),          # rows at negative positions
    ([300, 129], [301, 257], 1, 256, 128, "bf16"),
    ([513], [600], 2, 48, 48, "bf16"),                   # a page that is not a power of two
    ([260], [260], 1, 256, 256, "f32"),
]


@pytest.mark.parametrize("rows,lengths,H,D,ps,dtype", APPENDS)
@pytest.mark.parametrize("layout", ["slice", "heads first"])
def test_append_matches_the_definition(rows, lengths, H, D, ps, dtype, layout):
    u = Setup(lengths, H, D, ps, seed=sum(rows))
    rng = np.random.default_rng(1)
    T = sum(rows)
    # some heads stay below the scales held, some raise them
    gain = np.where(np.arange(H) % 2 == 0, 0.1, 6.0)[None, :, None]
    K, V = (strided((rng.standard_normal((T, H, D)) * gain).astype(F), dtype, 2, layout != "slice") for _ in range(2))
    off = None if set(rows) == {1} else offsets_of(rows)
    want = [plain_append(c, s, as_np(x), u.table, lengths, rows, ps)
            for c, s, x in ((u.kc, u.ks, K), (u.vc, u.vs, V))]
    for call in range(2):     # a second call of the same step changes nothing
        u.cache.append(K, V, u.len, u.pages, offsets=off, max_new=max(rows))
        got = [t.cpu().numpy() for t in u.dev]
        for g, w in zip(got, (want[0][0], want[0][1], want[1][0], want[1][1])):
            np.testing.assert_array_equal(g, w)
    assert u.cache.status() == mlora.MLORA_OK


def test_append_token_by_token_stays_within_a_step_of_the_value():
    """64 single tokens with growing size into one block: each growth quantises the block
    again, so a value may be off by half a step per growth that its code saw; here the size
    doubles four times: at most 1/2 + 1/2 (1 + 1/2 + 1/4 + ...) < 1.5 steps."""
    u = Setup([0], 2, 64, 64, seed=3, spare=2)
    table = torch.tensor([[1]], dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(4)
    x = rng.uniform(-1, 1, (64, 2, 64)).astype(F)
    x[:, :, 0] = 1.0                                   # the block's maximum is its first element's
    x *= (2.0 ** (np.arange(64) // 16))[:, None, None].astype(F)
    for t in range(64):
        k = torch.from_numpy(x[t:t + 1]).cuda()
        u.cache.append(k, k, torch.tensor([t + 1], dtype=torch.int32, device="cuda"), table)
    codes, scale = u.dev[0].cpu().numpy()[1], u.dev[1].cpu().numpy()[1]
    np.testing.assert_allclose(scale, 8.0 / 127, rtol=1e-6)
    back = codes.transpose(1, 0, 2).astype(np.float64) * scale[None, :, None]
    assert np.abs(back - x).max() <= 1.5 * scale.max()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_of_extreme_values(dtype):
    u = Setup([40], 4, 16, 64, seed=5)
    x = np.random.default_rng(6).standard_normal((40, 4, 16)).astype(F)
    x[3, 0, 5], x[4, 0, 6], x[5, 0, 7] = np.inf, -np.inf, np.nan
    x[:, 1] = 0.0
    x[:, 2] *= F(1e-39)                                # below the smallest scale: zeros
    x[:, 3] *= F(1e37)
    K = strided(x, dtype)
    want = plain_append(u.kc, u.ks, as_np(K), u.table, [40], [40], 64)
    u.cache.append(K, K, u.len, u.pages, offsets=offsets_of([40]), max_new=40)
    codes, scale = u.dev[0].cpu().numpy(), u.dev[1].cpu().numpy()
    np.testing.assert_array_equal(codes, want[0])
    np.testing.assert_array_equal(scale, want[1])
    page = u.table[0, 0]
    assert codes[page, 0, 3, 5] == 127 and codes[page, 0, 4, 6] == -127 and codes[page, 0, 5, 7] == 0
    assert not codes[page, 1, :40].any() and not codes[page, 2, :40].any() and scale[page, 1] == 0


# ---- read ------------------------------------------------------------------ #
@pytest.mark.parametrize("rows,lengths,H,D,ps,dtype", APPENDS)
def test_read_restores_values(rows, lengths, H, D, ps, dtype):
    u = Setup(lengths, H, D, ps, seed=8)
    T = sum(rows)
    out = [torch.full((T, H + 1, D), 7.0, dtype=TDT[dtype], device="cuda") for _ in range(2)]
    off = None if set(rows) == {1} else offsets_of(rows)
    u.cache.read(out[0][:, :H], out[1][:, 1:], u.len, u.pages, offsets=off, max_new=max(rows))
    for got, codes, scale in ((out[0][:, :H], u.kc, u.ks), (out[1][:, 1:], u.vc, u.vs)):
        want = [np.concatenate([np.zeros((max(0, n - length), H, D), F),
                                u.values(codes, scale, b, F)[max(0, length - n):]])
                for b, (n, length) in enumerate(zip(rows, lengths))]
        want = torch.from_numpy(np.concatenate(want)).to(TDT[dtype])
        assert torch.equal(got.cpu(), want)
    assert torch.all(out[0][:, H] == 7.0) and torch.all(out[1][:, 0] == 7.0)
    assert u.cache.status() == mlora.MLORA_OK


# ---- attend ---------------------------------------------------------------- #
def plain_attend(u, q, rows, scale, window):
    """(o, tolerance scale A, S per row) in 64 bits."""
    T, Hq, D = q.shape
    G = Hq // u.H
    o, A, S = np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.zeros((T, Hq, 1))
    at = 0
    for b, n in enumerate(rows):
        k, v = u.values(u.kc, u.ks, b), u.values(u.vc, u.vs, b)
        for i in range(n):
            pos = u.lengths[b] - n + i
            lo = max(0, pos - window + 1) if window else 0
            if pos < 0:
                continue
            kk, vv = k[lo:pos + 1], v[lo:pos + 1]
            for h in range(u.H):
                qh = q[at + i, h * G:(h + 1) * G].astype(np.float64)
                with np.errstate(all="ignore"):
                    x = scale * qh @ kk[:, h].T
                    p = np.exp(x - x.max(axis=1, keepdims=True))
                    p /= p.sum(axis=1, keepdims=True)
                    o[at + i, h * G:(h + 1) * G] = p @ vv[:, h]
                    A[at + i, h * G:(h + 1) * G] = p @ np.abs(vv[:, h])
                    S[at + i, h * G:(h + 1) * G] = (scale * np.abs(qh) @ np.abs(kk[:, h]).T).max(axis=1, keepdims=True)
        at += n
    return o, A, S


def tolerance(o, A, S, dtype):
    if dtype == "f32":
        return 2.0 ** -16 * (1 + S) * A + 1e-30
    return 2.0 ** -8 * np.abs(o) + (2.0 ** -7 + 2.0 ** -15 * (1 + S)) * A + 1e-30


def check_attend(u, rows, dtype, window=0, seed=11, q_size=1.0, scale=None, q=None, sliced=True):
    T = sum(rows)
    rng = np.random.default_rng(seed)
    if q is None:
        q = (rng.standard_normal((T, u.Hq, u.D)) * q_size).astype(F)
    Q = strided(q, dtype, 3 if sliced else 0)
    wide = torch.full((T, u.Hq + 1, u.D), 5.0, dtype=TDT[dtype], device="cuda")
    off = None if rows and set(rows) == {1} else offsets_of(rows)
    u.cache.attend(Q, wide[:, :u.Hq], u.len, u.pages, offsets=off, max_new=max(rows), scale=scale, window=window)
    got = as_np(wide[:, :u.Hq]).astype(np.float64)
    o, A, S = plain_attend(u, as_np(Q), rows, u.D ** -0.5 if scale is None else scale, window)
    bad = ~(np.abs(got - o) <= tolerance(o, A, S, dtype))
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.abs(got - o)[bad].max()}, first {np.argwhere(bad)[0]}"
    assert torch.all(wide[:, u.Hq] == 5.0)
    assert u.cache.status() == mlora.MLORA_OK
    return wide[:, :u.Hq]


ATTENDS = [
    # rows, lengths, H, G, D, page, window
    ([1], [1], 1, 1, 16, 16, 0),                               # a single token
    ([1, 1, 1], [15, 16, 17], 2, 1, 64, 16, 0),                # around a page's end
    ([1, 1, 1, 1, 1], [31, 0, 65, 1, 500], 2, 4, 128, 64, 0),  # an empty slot
    ([1] * 3, [1000, 2047, 3], 1, 8, 128, 32, 0),
    ([1, 1], [700, 90], 2, 7, 80, 48, 0),
    ([1, 1], [2500, 4100], 1, 16, 128, 128, 0),
    ([1], [5000], 1, 3, 256, 16, 0),                           # few heads: the long axis is split
    ([1, 1], [900, 40], 1, 71, 64, 16, 0),                     # one key head for many
    ([1, 1, 1], [300, 64, 65], 2, 2, 96, 64, 64),              # windows that end at a block's edge
    ([3, 1, 5], [3, 260, 77], 2, 4, 128, 64, 0),               # a few rows a sequence
    ([6, 2, 4], [2, 0, 4], 2, 2, 64, 16, 0),                   # rows at negative positions
    ([9, 0, 30], [1200, 8, 31], 1, 5, 64, 16, 33),
    ([130, 65, 7], [130, 300, 500], 2, 2, 128, 64, 0),         # prompts, some continued
    ([200], [200], 1, 1, 64, 16, 0),
    ([257, 1, 100], [257, 900, 1300], 1, 4, 128, 128, 0),      # a mixed batch
    ([150], [400], 2, 3, 80, 32, 100),
    ([140, 20], [290, 20], 1, 2, 256, 64, 0),
    ([129], [129], 1, 1, 112, 256, 17),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,lengths,H,G,D,ps,window", ATTENDS)
def test_attend_matches_64_bits(rows, lengths, H, G, D, ps, window, dtype):
    check_attend(Setup(lengths, H, D, ps, Hq=H * G, seed=9), rows, dtype, window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,lengths", [([1, 1], [777, 130]), ([140], [333])])
@pytest.mark.parametrize("q_size,k_size", [(30.0, 1.5), (1e-4, 1.5), (1e6, 1e-6), (1.0, 1e-30), (1e-20, 1e18)])
def test_attend_over_sizes_of_queries_and_keys(rows, lengths, q_size, k_size, dtype):
    """Peaked and flat softmax; queries outside fp16's range."""
    check_attend(Setup(lengths, 2, 128, 64, Hq=4, seed=10, k_size=k_size), rows, dtype, q_size=q_size)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size,others", [(1e30, 1.0), (1e-30, 1e-36), (1e-30, 0.0)])
@pytest.mark.parametrize("rows,lengths,D", [([1, 1, 1], [300, 64, 90], 128), ([131, 30], [200, 30], 128), ([40], [90], 64)])
def test_attend_over_unequal_query_rows(rows, lengths, D, size, others, dtype):
    """Every third row far outside the range of the rest, with keys that bring its scores to 1."""
    u = Setup(lengths, 1, D, 64, Hq=2, seed=25, k_size=1.0 / size)
    q = np.random.default_rng(26).standard_normal((sum(rows), 2, D)).astype(F) * F(others)
    q[::3] = (np.random.default_rng(27).standard_normal(q[::3].shape) * size).astype(F)
    check_attend(u, rows, dtype, q=q)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,lengths", [([1, 1], [520, 64]), ([130], [450])])
def test_attend_over_unequal_value_blocks(rows, lengths, dtype):
    """Scales of value blocks over twelve decades, among them zeros."""
    u = Setup(lengths, 1, 64, 16, Hq=2, seed=12)
    rng = np.random.default_rng(13)
    u.vs = np.where(np.isnan(u.vs), u.vs, 10.0 ** rng.uniform(-10, 2, u.vs.shape)).astype(F)
    u.vs[u.table[0, 1]] = 0.0
    u.ks[u.table[0, 2]] = 0.0
    u.upload()
    check_attend(u, rows, dtype)


@pytest.mark.parametrize("rows,lengths", [([1, 1, 1], [100, 30, 64]), ([131, 40], [200, 40])])
def test_attend_keeps_bad_queries_to_their_rows(rows, lengths):
    """A row whose query holds NaN or an infinity gives what it gives; the others are untouched."""
    u = Setup(lengths, 1, 128, 64, Hq=2, seed=14)
    q = np.random.default_rng(15).standard_normal((sum(rows), 2, 128)).astype(F)
    clean = check_attend(u, rows, "bf16", q=q).clone()
    q[1, 0, 3], q[0, 1, 7] = np.nan, np.inf
    Q = strided(q, "bf16")
    O = torch.empty_like(Q)
    u.cache.attend(Q, O, u.len, u.pages, offsets=offsets_of(rows), max_new=max(rows))
    assert torch.isnan(O[1, 0]).all() and not torch.isfinite(O[0, 1]).any()
    keep = torch.ones(Q.shape[:2], dtype=torch.bool, device="cuda")
    keep[1, 0] = keep[0, 1] = False
    assert torch.equal(O[keep], clean[keep])


@pytest.mark.parametrize("rows,lengths,G,D,dtype", [
    ([1] * 4, [3000, 17, 0, 900], 4, 128, "bf16"), ([3, 2], [2000, 600], 4, 64, "f32"),
    ([200, 65], [700, 65], 2, 128, "bf16"), ([1], [20000], 2, 128, "bf16")])
def test_attend_twice_gives_the_same_bits(rows, lengths, G, D, dtype):
    u = Setup(lengths, 2, D, 64, Hq=2 * G, seed=16)
    q = strided(np.random.default_rng(17).standard_normal((sum(rows), 2 * G, D)).astype(F), dtype)
    out = [torch.empty_like(q) for _ in range(3)]
    for o in out:
        u.cache.attend(q, o, u.len, u.pages, offsets=offsets_of(rows), max_new=max(rows))
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])


def test_attend_ignores_what_lies_past_the_length():
    """Codes past the length, and pages past the table's used part, do not matter."""
    u = Setup([70, 33], 2, 64, 32, Hq=4, seed=18)
    a = check_attend(u, [1, 1], "bf16").clone()
    u.kc[u.table[0, 2], :, 6:] = 127
    u.vc[u.table[0, 2], :, 6:] = -128
    u.vc[u.table[1, 1], :, 1:] = -128
    u.upload()
    assert torch.equal(a, check_attend(u, [1, 1], "bf16"))


def test_shared_pages_are_read_by_many():
    """Two sequences over the same prefix pages."""
    u = Setup([96, 96], 1, 64, 32, Hq=1, seed=19)
    u.table[1] = u.table[0]
    u.upload()
    q = np.random.default_rng(20).standard_normal((1, 1, 64)).astype(F)
    o = check_attend(u, [1, 1], "bf16", q=np.concatenate([q, q]))
    assert torch.equal(o[0], o[1])


# ---- steps out of range ---------------------------------------------------- #
def test_out_of_range_steps_are_reported_and_touch_nothing_else():
    u = Setup([40, 40, 40], 2, 64, 16, Hq=2, seed=21)
    before = [t.clone() for t in u.dev]
    rows = torch.randn((3, 2, 64), device="cuda").bfloat16()
    out = torch.full_like(rows, 3.0)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
    good = dict(lengths=u.len, pages=u.pages, offsets=i32([0, 1, 2, 3]))

    def calls(**kw):
        a = {**good, **kw}
        u.cache.append(rows, rows, a["lengths"], a["pages"], offsets=a["offsets"])
        u.cache.attend(rows, out, a["lengths"], a["pages"], offsets=a["offsets"])
        assert u.cache.status() == mlora.MLORA_ERR_DEVICE_STEP
        assert u.cache.status() == mlora.MLORA_OK     # read and cleared

    bad_page = u.pages.clone()
    bad_page[1, 2] = u.n_pages
    calls(pages=bad_page)
    page = int(u.table[1, 2])
    assert torch.equal(u.dev[0][page], before[0][page])        # nothing was stored for sequence 1
    bad_page[1, 2] = -1
    calls(pages=bad_page)
    calls(lengths=i32([40, 49, 40]))                           # more than the table holds
    calls(lengths=i32([40, -3, 40]))
    assert torch.all(out[1] == 0)
    out.fill_(3.0)
    calls(offsets=i32([0, 1, 7, 3]))                           # past T, then decreasing
    assert torch.all(out[1:] == 3.0)
    calls(offsets=i32([0, 0, 0, 3]))                           # more rows than max_new
    for t, old in zip(u.dev, before):                          # pages of nobody are untouched
        spare = [p for p in range(u.n_pages) if p not in u.table]
        assert torch.equal(t[spare].nan_to_num(), old[spare].nan_to_num())


def test_tokens_of_a_bad_page_read_as_zero():
    u = Setup([64, 20], 1, 64, 16, Hq=2, seed=22)
    keep = u.table.copy()
    u.table[0, 2] = u.n_pages + 5
    u.pages = torch.from_numpy(u.table).cuda()
    q = torch.randn((2, 2, 64), device="cuda")
    o = torch.empty_like(q)
    u.cache.attend(q, o, u.len, u.pages)
    k = torch.empty((64, 1, 64), device="cuda")
    v = torch.empty_like(k)
    u.cache.read(k, v, u.len[:1], u.pages[:1], offsets=offsets_of([64]), max_new=64)
    assert u.cache.status() == mlora.MLORA_ERR_DEVICE_STEP
    assert not k[32:48].any() and k[48:].any() and not v[32:48].any()
    u.table = keep
    page = keep[0, 2]
    u.kc[page] = u.vc[page] = 0
    want, A, S = plain_attend(u, as_np(q), [1, 1], 0.125, 0)
    assert (np.abs(as_np(o) - want) <= tolerance(want, A, S, "f32")).all()


def test_refusals():
    u = Setup([20, 5], 2, 64, 16, Hq=4, seed=23)
    k = torch.zeros((2, 2, 64), device="cuda", dtype=torch.bfloat16)
    q = torch.zeros((2, 4, 64), device="cuda", dtype=torch.bfloat16)
    for bad in (lambda: u.cache.append(k, k.float(), u.len, u.pages),
                lambda: u.cache.append(k.half(), k.half(), u.len, u.pages),
                lambda: u.cache.append(q, q, u.len, u.pages),
                lambda: u.cache.attend(k, k, u.len, u.pages),
                lambda: u.cache.append(k.transpose(1, 2).contiguous().transpose(1, 2), k, u.len, u.pages),
                lambda: u.cache.append(k, k, u.len.long(), u.pages),
                lambda: u.cache.append(k, k, u.len, u.pages.long()),
                lambda: u.cache.append(k, k, u.len[:1], u.pages),
                lambda: u.cache.append(k, k, u.len, u.pages, offsets=u.len),
                lambda: u.cache.append(k.cpu(), k.cpu(), u.len, u.pages),
                lambda: u.cache.append(k, k, u.len.cpu(), u.pages),
                lambda: Cache(u.dev[0].float(), *u.dev[1:], 4),
                lambda: Cache(u.dev[0], u.dev[1][:1], *u.dev[2:], 4),
                lambda: Cache(u.dev[0].cpu(), *u.dev[1:], 4)):
        with pytest.raises(ValueError):
            bad()
    odd = torch.zeros((2, 2 * 64 + 4), device="cuda", dtype=torch.bfloat16)
    for bad in (lambda: u.cache.append(odd[:, 4:].unflatten(1, (2, 64)), k, u.len, u.pages),
                lambda: u.cache.append(torch.cat([k, k]), torch.cat([k, k]), u.len, u.pages),   # T, no offsets
                lambda: u.cache.attend(q, q.clone(), u.len, u.pages, scale=0.0),
                lambda: u.cache.attend(q, q.clone(), u.len, u.pages, scale=math.nan),
                lambda: u.cache.attend(q, q.clone(), u.len, u.pages, window=-1),
                lambda: u.cache.append(k, k, u.len, u.pages, max_new=-1)):
        with pytest.raises(mlora.MloraError) as e:
            bad()
        assert e.value.status == mlora.MLORA_ERR_INVALID_ARG
    with pytest.raises(mlora.MloraError) as e:
        Cache(*u.dev, 3)
    assert e.value.status == mlora.MLORA_ERR_INVALID_ARG


def test_empty_steps_do_nothing():
    u = Setup([20], 2, 64, 16, seed=24)
    none = torch.zeros((0, 2, 64), device="cuda")
    before = [t.clone() for t in u.dev]
    u.cache.append(none, none, u.len[:0], u.pages[:0])
    u.cache.attend(none, none, u.len[:0], u.pages[:0])
    u.cache.append(none, none, u.len, u.pages, offsets=offsets_of([0]), max_new=0)
    u.cache.attend(none, none, u.len, u.pages, offsets=offsets_of([0]), max_new=4)
    assert all(torch.equal(a.nan_to_num(), b.nan_to_num()) for a, b in zip(u.dev, before))
    assert u.cache.status() == mlora.MLORA_OK


# ---- streams, graphs, large offsets ---------------------------------------- #
def test_a_step_on_another_stream_and_in_a_graph():
    u = Setup([100, 40], 2, 128, 16, Hq=4, seed=25)
    rng = np.random.default_rng(26)
    K, V = (strided(rng.standard_normal((2, 2, 128)).astype(F), "bf16") for _ in range(2))
    Q = strided(rng.standard_normal((2, 4, 128)).astype(F), "bf16")
    want = torch.empty_like(Q)
    u.cache.append(K, V, u.len, u.pages)
    u.cache.attend(Q, want, u.len, u.pages)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = torch.zeros_like(Q)
    side.wait_stream(torch.cuda.current_stream())
    u.cache.append(K, V, u.len, u.pages, stream=side)
    u.cache.attend(Q, got, u.len, u.pages, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    got.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        u.cache.append(K, V, u.len, u.pages)
        u.cache.attend(Q, got, u.len, u.pages)
    for _ in range(2):
        got.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    assert u.cache.status(side) == mlora.MLORA_OK


def test_pages_past_32_bit_offsets():
    """Codes past 2^31 bytes of the page array (8.6 GB in all)."""
    H, ps, D, n_pages = 4, 128, 128, 65600
    kc, vc = (torch.zeros((n_pages, H, ps, D), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((n_pages, H), float("nan"), device="cuda") for _ in range(2))
    cache = Cache(kc, ks, vc, vs, 8)
    table = torch.tensor([[65599, 40000], [0, 65590]], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    K, V = (torch.randn((400, H, D), device="cuda", generator=g) for _ in range(2))
    length = torch.tensor([200, 200], dtype=torch.int32, device="cuda")
    cache.append(K, V, length, table, offsets=offsets_of([200, 200]), max_new=200)
    for t in (65599, 40000, 0, 65590):
        assert torch.isfinite(ks[t]).all() and torch.count_nonzero(kc[t]) > 0
    rk, rv = torch.empty_like(K), torch.empty_like(V)
    cache.read(rk, rv, length, table, offsets=offsets_of([200, 200]), max_new=200)
    assert (rk - K).abs().max() <= 0.51 * ks[[65599, 40000, 0, 65590]].max()
    Q = torch.randn((2, 8, D), device="cuda", generator=g)
    O = torch.empty_like(Q)
    cache.attend(Q, O, length, table)
    for b in range(2):
        k, v = (x[200 * b:200 * b + 200].double().repeat_interleave(2, dim=1) for x in (rk, rv))
        w = torch.einsum("hd,thd->ht", Q[b].double(), k) * D ** -0.5
        want = torch.einsum("ht,thd->hd", w.softmax(-1), v)
        assert (O[b] - want).abs().max() < 1e-3 * want.abs().max()
    assert cache.status() == mlora.MLORA_OK


def test_prompts_converted_once_or_in_place_give_the_same_bits():
    """Room for all, one, or none of a step's sequences in the workspace for prompts."""
    rows, lengths = [400, 300, 70, 512], [900, 300, 333, 512]
    u = Setup(lengths, 2, 128, 64, Hq=4, seed=27)
    q = strided(np.random.default_rng(28).standard_normal((sum(rows), 4, 128)).astype(F), "bf16")
    tile = 128 * 2 * 128 * 4                                  # bytes of 128 tokens, two heads
    outs = []
    for room in (256 << 20, 9 * tile, 0):
        cache = Cache(*u.dev, 4, prompt_bytes=room)
        for window in (0, 200):
            o = torch.full_like(q, float("nan"))
            cache.attend(q, o, u.len, u.pages, offsets=offsets_of(rows), max_new=max(rows), window=window)
            outs.append(o)
        assert cache.status() == mlora.MLORA_OK
    for k in (2, 4):
        assert torch.equal(outs[0], outs[k]) and torch.equal(outs[1], outs[k + 1])


@pytest.mark.parametrize("D,ps,dtype", [(128, 64, "bf16"), (64, 16, "bf16"), (80, 48, "bf16"), (256, 32, "bf16"),
                                        (128, 128, "f32"), (48, 16, "f32")])
@pytest.mark.parametrize("window", [0, 150])
def test_long_prompts_converted_once_or_in_place(D, ps, dtype, window):
    """More rows than are converted in place: room for all, for the first, or for none of the sequences."""
    rows, lengths = [250, 60, 410], [250, 500, 700]
    u = Setup(lengths, 1, D, ps, Hq=16, seed=31)
    outs = []
    for room in (256 << 20, 140000 * (64 if D <= 64 else 128 if D <= 128 else 256) // 128, 0):
        u.cache = Cache(*u.dev, 16, prompt_bytes=room)
        outs.append(check_attend(u, rows, dtype, window).clone())
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("rows,lengths,H,G,D,ps,window", [
    ([20], [3000], 1, 1, 128, 64, 0),                          # few row tiles: their tokens in parts
    ([40, 3], [2000, 700], 1, 4, 64, 16, 0),
    ([20, 20, 1], [1100, 20, 0], 2, 2, 256, 32, 0),
    ([300], [2000], 1, 1, 256, 128, 500),
    ([5], [5000], 1, 8, 192, 48, 0),
    ([70], [4500], 1, 2, 80, 64, 3000),
    ([33], [40], 1, 1, 160, 16, 0),
])
@pytest.mark.parametrize("room", [256 << 20, 0])
def test_prompts_in_parts_and_wide_heads(rows, lengths, H, G, D, ps, window, room):
    u = Setup(lengths, H, D, ps, Hq=H * G, seed=29)
    u.cache = Cache(*u.dev, H * G, prompt_bytes=room)
    first = check_attend(u, rows, "bf16", window)
    assert torch.equal(first, check_attend(u, rows, "bf16", window))


def test_long_sums_of_fp32_rows_keep_their_bits():
    """Values of one sign over many tokens, as many items as CTAs, so that each sums a long range.  A
    sum of n / 16 parts rounded to nearest is off by some sqrt(n / 16) 2^-24 of it, here 1.9e-6;
    sums that drop bits instead are off by n / 16 of half of them."""
    B, H, D, ps, n = 152, 2, 64, 64, 16000
    rng = np.random.default_rng(32)
    kc = torch.from_numpy(rng.integers(-127, 128, (n // ps, H, ps, D)).astype(np.int8)).cuda()
    vc = torch.from_numpy(rng.integers(60, 128, (n // ps, H, ps, D)).astype(np.int8)).cuda()
    ks, vs = (torch.full((n // ps, H), 0.01, device="cuda") for _ in range(2))
    cache = Cache(kc, ks, vc, vs, H)
    q = torch.from_numpy((rng.standard_normal((B, H, D)) * 0.3).astype(F)).cuda()
    o = torch.empty_like(q)
    lengths = torch.full((B,), n, dtype=torch.int32, device="cuda")
    pages = torch.arange(n // ps, dtype=torch.int32, device="cuda").expand(B, -1).contiguous()   # shared by all
    cache.attend(q, o, lengths, pages)
    k = (kc.double() * ks.double()[:, :, None, None]).permute(1, 0, 2, 3).reshape(H, n, D)
    v = (vc.double() * vs.double()[:, :, None, None]).permute(1, 0, 2, 3).reshape(H, n, D)
    p = torch.softmax(D ** -0.5 * torch.einsum("bhd,hnd->bhn", q.double(), k), dim=2)
    want = torch.einsum("bhn,hnd->bhd", p, v)
    assert (o.double() - want).norm() < 2.0 ** -18 * want.norm()
    assert cache.status() == mlora.MLORA_OK


def test_long_sums_of_fp32_prompts_keep_their_bits():
    """The same for prompts: sums that cut off in the tensor cores, of 1024 tokens at most, lose at most
    2^-23 of the sum so far at each of 64 steps, 2^-18 of the whole."""
    B, R, D, ps, n = 152, 20, 64, 64, 16000
    rng = np.random.default_rng(33)
    kc = torch.from_numpy(rng.integers(-127, 128, (n // ps, 1, ps, D)).astype(np.int8)).cuda()
    vc = torch.from_numpy(rng.integers(60, 128, (n // ps, 1, ps, D)).astype(np.int8)).cuda()
    ks, vs = (torch.full((n // ps, 1), 0.01, device="cuda") for _ in range(2))
    cache = Cache(kc, ks, vc, vs, 1)
    q = torch.from_numpy((rng.standard_normal((B * R, 1, D)) * 0.3).astype(F)).cuda()
    o = torch.full_like(q, float("nan"))
    lengths = torch.full((B,), n, dtype=torch.int32, device="cuda")
    pages = torch.arange(n // ps, dtype=torch.int32, device="cuda").expand(B, -1).contiguous()
    cache.attend(q, o, lengths, pages, offsets=offsets_of([R] * B), max_new=R)
    k = (kc.double() * ks.double()[:, :, None, None]).reshape(n, D)
    v = (vc.double() * vs.double()[:, :, None, None]).reshape(n, D)
    pos = n - R + torch.arange(B * R, device="cuda") % R
    x = D ** -0.5 * q[:, 0].double() @ k.T
    x = x.masked_fill(torch.arange(n, device="cuda")[None] > pos[:, None], -float("inf"))
    want = torch.softmax(x, dim=1) @ v
    assert (o[:, 0].double() - want).norm() < 2.0 ** -18 * want.norm()
    assert cache.status() == mlora.MLORA_OK


def test_growing_scores_move_the_bound():
    """Keys that grow along the sequence: the softmax bound moves in the middle of it, for some
    rows and not for others."""
    for rows, lengths, G in (([1], [4000], 2), ([150], [1000], 2), ([20], [3000], 1)):
        u = Setup(lengths, 1, 128, 64, Hq=G, seed=30, k_size=0.02)
        for j in range(u.table.shape[1]):
            u.ks[u.table[0, j]] *= F(1.25 ** min(j, 30))
        u.upload()
        check_attend(u, rows, "bf16", q_size=2.0)
        check_attend(u, rows, "f32", q_size=2.0)
