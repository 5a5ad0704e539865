"""The 4-bit key/value cache and its attention through the public entry points, against plain
implementations: blocks byte for byte (the definition's fp32 operations in numpy), attention in
64 bits.  The tolerances are test_gpu_cache.py's, whose derivation holds here: a code times its
scale is exact in the products' operands, so that weights, sums and the output are what rounds.
One term more: up to 16 rows a sequence and key head, weights are fp16 numbers of which a row's
largest is 2^12 or more, so that each is also off by up to 2^-25: 2^-37 of the weights' sum.  It
shows where a token holds a zero, as one in 15 codes is, and nearly all of the weight."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():   # pragma: no cover - CPU machine
    pytest.skip("needs a GPU", allow_module_level=True)

from heterogeneous_lora_gemm_gb300 import Cache4, mlora  # noqa: E402
from test_gpu_cache import (APPENDS, ATTENDS, F, TDT, as_np, offsets_of, plain_attend,  # noqa: E402
                            strided, tolerance)

# e4m3 without its sign: bytes 0 .. 126
E4M3 = np.array([(1 + m / 8) * 2.0 ** (e - 7) if e else m * 2.0 ** -9 for e in range(16) for m in range(8)][:127])


def atoms(D):
    """Number of the atom of token t and group g in a block: ([16, D / 16] of keys, of values)."""
    n = D // 16
    t, g = np.arange(16)[:, None], np.arange(n)[None]
    k = g // 4 * 64 + (t % 8 * np.minimum(4, n - g // 4 * 4) + g % 4) * 2 + t // 8
    v = g // 8 * 128 + (t // 8 * np.minimum(8, n - g // 8 * 8) + g % 8) * 8 + t % 8
    return k, v


def unpack(blocks, keys):
    """Codes [..., 16, D] and scale bytes [..., 16, D / 16] of blocks [..., 18 D]."""
    D = blocks.shape[-1] // 18
    at = atoms(D)[0 if keys else 1]
    first = 0 if keys else 8 * D
    w = blocks[..., first:first + 8 * D].reshape(blocks.shape[:-1] + (D, 8))[..., at, :]
    codes = np.stack([w & 15, w >> 4], axis=-1).reshape(blocks.shape[:-1] + (16, D)).astype(np.int8) - 8
    return codes, blocks[..., (16 if keys else 17) * D:][..., :D][..., at]


def pack(blocks, keys, codes, scales):
    """The reverse, into blocks."""
    D = blocks.shape[-1] // 18
    at = atoms(D)[0 if keys else 1]
    n = (codes + 8).astype(np.uint8).reshape(codes.shape[:-1] + (D // 16, 8, 2))
    first = 0 if keys else 8 * D
    w = blocks[..., first:first + 8 * D].reshape(blocks.shape[:-1] + (D, 8))
    w[..., at, :] = n[..., 0] | n[..., 1] << 4
    blocks[..., first:first + 8 * D] = w.reshape(blocks.shape[:-1] + (8 * D,))
    s = blocks[..., (16 if keys else 17) * D:(17 if keys else 18) * D]
    s[..., at] = scales


class Setup4:
    """Blocks with random codes and scales in their tokens, random bytes everywhere else, shuffled page tables."""

    def __init__(self, lengths, H, D, ps, Hq=None, seed=0, spare=3, k_unit=0.05, v_unit=0.02, scales=None, room=256 << 20, width=1):
        rng = np.random.default_rng(seed)
        self.lengths, self.H, self.D, self.ps, self.Hq = list(lengths), H, D, ps, Hq or H
        self.units, self.room = (k_unit, v_unit), room
        used = [-(-max(n, 0) // ps) for n in lengths]
        self.n_pages = sum(used) + spare
        order = rng.permutation(self.n_pages)
        self.width = max([width] + used)      # (entries past the sequences' blocks are never read)
        self.table = np.full((len(lengths), self.width), -7, np.int32)   # unused entries are never read
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = order[at:at + u]
            at += u
        self.blocks = rng.integers(0, 256, (self.n_pages, H, ps // 16, 18 * D)).astype(np.uint8)
        self.kc, self.vc, self.ks, self.vs = True, False, None, None    # (as plain_attend asks for values)
        codes = self.held(lambda shape: rng.integers(-7, 8, shape).astype(np.int8),
                          scales or (lambda shape: rng.integers(44, 64, shape)))
        self.fill(*codes)
        self.upload()

    def held(self, codes, scales):
        """Codes and scale bytes of the keys and values of every token slot: (kc, ks, vc, vs)."""
        shape = (self.n_pages, self.H, self.ps // 16, 16)
        return sum(((codes(shape + (self.D,)), scales(shape + (self.D // 16,))) for _ in range(2)), ())

    def fill(self, kc, ks, vc, vs):
        """Into the tokens that the sequences hold; the other bytes stay."""
        whole = self.blocks.copy()
        pack(whole, True, kc, ks)
        pack(whole, False, vc, vs)
        mine = np.zeros(self.blocks.shape, bool)
        for t, n in zip(self.table, self.lengths):
            for j in range(-(-max(n, 0) // 16)):
                live = np.arange(16) < n - j * 16
                one = np.zeros(18 * self.D, bool)
                for a, first, scale in zip(atoms(self.D), (0, 8 * self.D), (16 * self.D, 17 * self.D)):
                    a = a[live].ravel()
                    one[(first + a[:, None] * 8 + np.arange(8)).ravel()] = True
                    one[scale + a] = True
                page, i = divmod(j * 16, self.ps)
                mine[t[page], :, i // 16] |= one
        self.blocks = np.where(mine, whole, self.blocks)
        self.mine = mine

    def upload(self):
        self.dev = torch.from_numpy(self.blocks).cuda()
        self.pages = torch.from_numpy(self.table).cuda()
        self.len = torch.tensor(self.lengths, dtype=torch.int32, device="cuda")
        self.cache = Cache4(self.dev, self.Hq, *self.units, prompt_bytes=self.room)

    def values(self, keys, _, b, dtype=np.float64):
        """[length, H, D] that sequence b holds."""
        n = self.lengths[b]
        t = self.table[b, :-(-n // self.ps)]
        codes, scales = unpack(self.blocks[t], keys)
        unit = F(self.units[0 if keys else 1])
        x = codes.reshape(scales.shape + (16,)) * np.append(E4M3, 0)[np.minimum(scales, 127)].astype(dtype)[..., None]
        x = (x.astype(dtype) * dtype(unit)).reshape(codes.shape)         # (the first product is exact)
        return x.transpose(0, 2, 3, 1, 4).reshape(-1, self.H, self.D)[:n]


# ---- append ---------------------------------------------------------------- #
def e4m3_of(x):
    """Bytes of fp32 numbers >= 0, to nearest, ties to even, at most 448."""
    x = np.minimum(x.astype(np.float64), 448.0)
    d = np.abs(x[..., None] - E4M3)
    best = d.min(-1, keepdims=True) == d
    even = best & (np.arange(127) % 2 == 0)
    return np.where(best.sum(-1) > 1, even.argmax(-1), best.argmax(-1)).astype(np.uint8)


def quantised(x, unit):
    """Codes and scale bytes of rows [..., D] by the definition, in fp32."""
    unit = F(unit)
    g = x.astype(F).reshape(x.shape[:-1] + (-1, 16))
    with np.errstate(all="ignore"):
        top = np.abs(np.where(np.isfinite(g), g, F(0))).max(-1)
        s = e4m3_of(top * (F(1) / (F(7) * unit)))
        step = E4M3[s].astype(F) * unit
        inv = np.where(s > 0, F(1) / step, F(0))
        q = g * inv[..., None]
        q = np.where(np.isnan(q), F(0), np.clip(q, F(-7), F(7)))
    return np.rint(q).astype(np.int8).reshape(x.shape), s


def plain_append(u, x, rows, keys):
    """u.blocks after the step."""
    codes, scales = unpack(u.blocks, keys)
    at = 0
    for b, (n, length) in enumerate(zip(rows, u.lengths)):
        for i in range(n):
            pos = length - n + i
            if pos >= 0:
                place = u.table[b, pos // u.ps], slice(None), pos % u.ps // 16, pos % 16
                codes[place], scales[place] = quantised(x[at + i], u.units[0 if keys else 1])
        at += n
    out = u.blocks.copy()
    pack(out, keys, codes, scales)
    return out


@pytest.mark.parametrize("rows,lengths,H,D,ps,dtype", APPENDS + [
    ([8, 3, 1], [9, 40, 1], 5, 208, 16, "bf16"), ([9, 3, 17], [9, 40, 33], 3, 16, 48, "f32")])
@pytest.mark.parametrize("layout", ["slice", "heads first"])
def test_append_matches_the_definition(rows, lengths, H, D, ps, dtype, layout):
    u = Setup4(lengths, H, D, ps, seed=sum(rows))
    rng = np.random.default_rng(1)
    T = sum(rows)
    gain = np.where(np.arange(H) % 2 == 0, 0.01, 6.0)[None, :, None]
    K, V = (strided((rng.standard_normal((T, H, D)) * gain).astype(F), dtype, 2, layout != "slice") for _ in range(2))
    off = None if set(rows) == {1} else offsets_of(rows)
    u.blocks = plain_append(u, as_np(K), rows, True)
    u.blocks = plain_append(u, as_np(V), rows, False)
    for call in range(2):     # a second call of the same step changes nothing
        u.cache.append(K, V, u.len, u.pages, offsets=off, max_new=max(rows))
        np.testing.assert_array_equal(u.dev.cpu().numpy(), u.blocks)
    assert u.cache.status() == mlora.MLORA_OK


@pytest.mark.parametrize("rows", [5, 40])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_of_extreme_values(rows, dtype):
    """Infinities, NaN, zeros, and groups below, at and above the range of the scales."""
    u = Setup4([rows], 6, 32, 64, seed=5, k_unit=0.0625, v_unit=2.0 ** -60)
    x = np.random.default_rng(6).standard_normal((rows, 6, 32)).astype(F)
    x[2, 0, 5], x[3, 0, 6], x[4, 0, 7] = np.inf, -np.inf, np.nan
    x[1, 0, 16:] = np.inf
    x[:, 1] = 0.0
    x[:, 2] *= F(1e-39)
    x[:, 3] *= F(1e37)
    x[:, 4] *= (10.0 ** np.linspace(-5, 5, rows))[:, None]
    x[:, 5] *= F(2.0 ** -10)
    K = strided(x, dtype)
    u.blocks = plain_append(u, as_np(K), [rows], True)
    u.blocks = plain_append(u, as_np(K), [rows], False)
    u.cache.append(K, K, u.len, u.pages, offsets=offsets_of([rows]), max_new=rows)
    np.testing.assert_array_equal(u.dev.cpu().numpy(), u.blocks)
    k = u.values(True, None, 0)
    assert k[2, 0, 5] > 0 and k[3, 0, 6] < 0 and k[4, 0, 7] == 0 and not k[1, 0, 16:].any() and not k[:, 1].any()
    assert np.abs(k[:, 3]).max() == F(0.0625) * 3136 and not k[:, 2].any()


def test_append_of_single_tokens_is_append_of_all():
    u, w = (Setup4([77], 2, 80, 32, seed=7) for _ in range(2))
    x = strided(np.random.default_rng(8).standard_normal((77, 2, 80)).astype(F), "bf16")
    u.cache.append(x, x, u.len, u.pages, offsets=offsets_of([77]), max_new=77)
    for t in range(77):
        w.cache.append(x[t:t + 1], x[t:t + 1], torch.tensor([t + 1], dtype=torch.int32, device="cuda"), w.pages)
    assert torch.equal(u.dev, w.dev)


# ---- read ------------------------------------------------------------------ #
@pytest.mark.parametrize("rows,lengths,H,D,ps,dtype", APPENDS + [([8, 3, 1], [9, 40, 1], 5, 208, 16, "bf16")])
def test_read_restores_values(rows, lengths, H, D, ps, dtype):
    u = Setup4(lengths, H, D, ps, seed=8)
    T = sum(rows)
    out = [torch.full((T, H + 1, D), 7.0, dtype=TDT[dtype], device="cuda") for _ in range(2)]
    off = None if set(rows) == {1} else offsets_of(rows)
    u.cache.read(out[0][:, :H], out[1][:, 1:], u.len, u.pages, offsets=off, max_new=max(rows))
    for got, keys in ((out[0][:, :H], True), (out[1][:, 1:], False)):
        want = [np.concatenate([np.zeros((max(0, n - length), H, D), F), u.values(keys, None, b, F)[max(0, length - n):]])
                for b, (n, length) in enumerate(zip(rows, lengths))]
        want = torch.from_numpy(np.concatenate(want)).to(TDT[dtype])
        assert torch.equal(got.cpu(), want)
    assert torch.all(out[0][:, H] == 7.0) and torch.all(out[1][:, 0] == 7.0)
    assert u.cache.status() == mlora.MLORA_OK


# ---- attend ---------------------------------------------------------------- #
def check_attend(u, rows, dtype, window=0, q_size=1.0, scale=None, q=None):
    T = sum(rows)
    if q is None:
        q = (np.random.default_rng(11).standard_normal((T, u.Hq, u.D)) * q_size).astype(F)
    Q = strided(q, dtype, 3)
    wide = torch.full((T, u.Hq + 1, u.D), 5.0, dtype=TDT[dtype], device="cuda")
    off = None if rows and set(rows) == {1} else offsets_of(rows)
    u.cache.attend(Q, wide[:, :u.Hq], u.len, u.pages, offsets=off, max_new=max(rows), scale=scale, window=window)
    got = as_np(wide[:, :u.Hq]).astype(np.float64)
    o, A, S = plain_attend(u, as_np(Q), rows, u.D ** -0.5 if scale is None else scale, window)
    low = np.zeros((T, 1, 1))
    at = np.concatenate([[0], np.cumsum(rows)])
    for b, n in enumerate(u.lengths):
        if n > 0:
            low[at[b]:at[b + 1]] = 2.0 ** -37 * n * np.abs(u.values(False, None, b)).max()
    bad = ~(np.abs(got - o) <= tolerance(o, A, S, dtype) + low)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.abs(got - o)[bad].max()}, first {np.argwhere(bad)[0]}"
    assert torch.all(wide[:, u.Hq] == 5.0)
    assert u.cache.status() == mlora.MLORA_OK
    return wide[:, :u.Hq]


@pytest.mark.parametrize("G", [1, 12, 20])
@pytest.mark.parametrize("D", [16, 64, 128, 256])
def test_every_scale_and_code_is_exact(D, G):
    """Sequences of one token, whose weight is 1: the output is the value.  (A value has 7 bits and so is
    exact in both types under a unit that is a power of two.)"""
    n = 127 * 15
    groups = D // 16
    u = Setup4([1] * (-(-n // groups)), 1, D, 16, Hq=G, seed=9, v_unit=0.5, k_unit=1.0)
    kc, ks, vc, vs = u.held(lambda s: np.zeros(s, np.int8), lambda s: np.full(s, 56))
    at = np.arange(u.table.shape[0] * groups) % n
    vs[u.table[:, 0], 0, 0, 0] = (at % 127).reshape(-1, groups)
    vc[u.table[:, 0], 0, 0, 0] = ((at // 127)[:, None] + np.arange(16)).reshape(-1, D) % 15 - 7
    u.fill(kc, ks, vc, vs)
    u.upload()
    for dtype in (torch.float32, torch.bfloat16):
        q = torch.randn((u.table.shape[0], G, D), device="cuda").to(dtype)
        o = torch.empty_like(q)
        u.cache.attend(q, o, u.len, u.pages)
        want = np.stack([u.values(False, None, b)[0, 0] for b in range(q.shape[0])])
        np.testing.assert_array_equal(o.double().cpu().numpy(), np.broadcast_to(want[:, None], o.shape))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,lengths,H,G,D,ps,window", ATTENDS + [
    ([1, 1], [70, 300], 2, 4, 48, 32, 0), ([2, 9], [70, 300], 1, 1, 208, 16, 50), ([30], [300], 1, 2, 144, 80, 0)])
def test_attend_matches_64_bits(rows, lengths, H, G, D, ps, window, dtype):
    check_attend(Setup4(lengths, H, D, ps, Hq=H * G, seed=9), rows, dtype, window)


def long_table(lengths, H, ps):
    """Columns of a page table of so many tokens that ranges are cut as for long sequences."""
    return 300000 // (len(lengths) * H * ps) + 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,lengths,H,G,D,ps,window", [case for case in ATTENDS if max(case[0]) * case[3] <= 16] + [
    ([1, 1], [70, 300], 2, 4, 48, 32, 0), ([1], [9000], 1, 8, 64, 16, 0), ([2, 1], [9000, 170], 1, 4, 128, 48, 700),
    ([1] * 600, [40] * 600, 4, 1, 64, 16, 0)])
def test_attend_under_page_tables_for_long_sequences(rows, lengths, H, G, D, ps, window, dtype):
    """Whatever of the tables the sequences use."""
    check_attend(Setup4(lengths, H, D, ps, Hq=H * G, seed=9, width=long_table(lengths, H, ps)), rows, dtype, window)


SHORT = [1, 31, 32, 33, 64, 65, 128, 129, 160, 256, 257, 288, 289, 512, 513, 0, 1000]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths,G,window", [([n], 4, 0) for n in SHORT if n] + [(SHORT, 1, 0), (SHORT, 4, 100),
                                              (SHORT * 8, 16, 0), (SHORT * 40, 2, 0), ([256] * 300, 4, 33)])
def test_items_of_few_chunks(lengths, G, window, dtype):
    """Below, at and past the lengths that one warp, one CTA and several take; fewer and more of them than
    there are CTAs; sequences of no token between."""
    check_attend(Setup4(lengths, 2, 64, 32, Hq=2 * G, seed=70), [1] * len(lengths), dtype, window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,lengths,D", [([1, 1], [777, 130], 128), ([140], [333], 128), ([3], [90], 256), ([40], [90], 64)])
@pytest.mark.parametrize("q_size,k_unit,v_unit", [(30.0, 0.05, 1.0), (1e-4, 0.05, 2.0 ** 60), (1e6, 1e-7, 2.0 ** -60),
                                                  (1.0, 2.0 ** -60, 1.0), (1e-18, 2.0 ** 60, 1.0), (1e-24, 2.0 ** 60, 1.0),
                                                  (3e6, 0.05, 1.0), (3e7, 0.05, 1.0)])
def test_attend_over_units_and_sizes_of_queries(rows, lengths, D, q_size, k_unit, v_unit, dtype):
    """Peaked and flat softmax; queries outside fp16's range; the units' limits."""
    u = Setup4(lengths, 2, D, 64, Hq=4, seed=10, k_unit=k_unit, v_unit=v_unit)
    check_attend(u, rows, dtype, q_size=q_size)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,lengths,D", [([1, 1], [300, 64], 128), ([131, 30], [200, 30], 128), ([3], [90], 64), ([9], [90], 256)])
def test_the_largest_queries(rows, lengths, D, dtype):
    """Rows up to 2^128 beside rows of 2^100, and a scale that brings the scores of the first to some tens."""
    u = Setup4(lengths, 1, D, 64, Hq=2, seed=58, k_unit=2.0 ** -60, scales=lambda shape: np.random.default_rng(1).integers(1, 12, shape))
    q = np.random.default_rng(59).uniform(-2.0 ** 100, 2.0 ** 100, (sum(rows), 2, D))
    q[::2] *= 2.0 ** 27.5
    check_attend(u, rows, dtype, q=q.astype(F), scale=2.0 ** -59)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,lengths,D", [([1, 1], [520, 64], 64), ([130], [450], 80), ([7], [700], 128), ([33, 2], [300, 100], 256)])
def test_attend_over_all_scales(rows, lengths, D, dtype):
    """Neighbouring groups and tokens with scales from 0 to 448."""
    rng = np.random.default_rng(12)
    u = Setup4(lengths, 1, D, 16, Hq=2, seed=12, k_unit=0.002, scales=lambda shape: rng.integers(0, 127, shape))
    check_attend(u, rows, dtype, q_size=0.3)


@pytest.mark.parametrize("rows,lengths", [([1, 1, 1], [100, 30, 64]), ([131, 40], [200, 40])])
def test_attend_keeps_bad_queries_to_their_rows(rows, lengths):
    u = Setup4(lengths, 1, 128, 64, Hq=2, seed=14)
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
    u = Setup4(lengths, 2, D, 64, Hq=2 * G, seed=16)
    q = strided(np.random.default_rng(17).standard_normal((sum(rows), 2 * G, D)).astype(F), dtype)
    out = [torch.empty_like(q) for _ in range(3)]
    for o in out:
        u.cache.attend(q, o, u.len, u.pages, offsets=offsets_of(rows), max_new=max(rows))
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,lengths,H,G,D,room", [
    ([1, 1, 1], [70, 33, 9], 2, 2, 64, 0), ([2, 5], [75, 5], 1, 3, 128, 0), ([1], [170], 1, 1, 256, 0), ([1], [90], 1, 1, 80, 0),
    ([40, 20], [70, 33], 1, 2, 128, 0), ([250, 60], [250, 500], 1, 16, 64, 256 << 20), ([30], [139], 1, 1, 208, 0)])
def test_bytes_that_nothing_was_written_to_do_not_matter(rows, lengths, H, G, D, room, dtype):
    """Among them scales that are not numbers, and those of the largest exponents."""
    u = Setup4(lengths, H, D, 48, Hq=H * G, seed=18, room=room)
    q = np.random.default_rng(19).standard_normal((sum(rows), H * G, D)).astype(F)
    first = check_attend(u, rows, dtype, q=q).clone()
    for byte in (0, 0x7F, 0xFF, 0x80, 0xFE):
        u.blocks = np.where(u.mine, u.blocks, byte).astype(np.uint8)
        u.upload()
        assert torch.equal(first, check_attend(u, rows, dtype, q=q))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("left", ["none", "bad"])
@pytest.mark.parametrize("rows,lengths,H,G,D,ps,window,room", [
    ([1, 1, 1], [300, 64, 65], 2, 2, 96, 16, 40, 0), ([1, 3], [1000, 700], 1, 4, 128, 32, 100, 0),
    ([1], [5000], 1, 3, 256, 16, 1000, 0), ([150, 20], [400, 300], 2, 3, 80, 32, 100, 0),
    ([40], [700], 1, 2, 128, 64, 130, 0), ([300], [2000], 1, 1, 256, 16, 500, 0),
    ([250, 60], [2250, 500], 1, 16, 128, 64, 150, 256 << 20)])
def test_pages_behind_the_window_are_not_read(rows, lengths, H, G, D, ps, window, room, left, dtype):
    """Their entries in the page table hold no page, or one of scales that are not numbers."""
    u = Setup4(lengths, H, D, ps, Hq=H * G, seed=51, room=room)
    free = next(p for p in range(u.n_pages) if p not in u.table)
    u.blocks[free] = 0xFF
    for t, n, length in zip(u.table, rows, lengths):
        t[:max(0, length - n - window + 1) // ps] = -1 if left == "none" else free
    u.upload()
    check_attend(u, rows, dtype, window)


@pytest.mark.parametrize("D,ps,dtype", [(128, 64, "bf16"), (64, 16, "bf16"), (80, 48, "bf16"), (256, 32, "bf16"),
                                        (128, 128, "f32"), (48, 16, "f32")])
@pytest.mark.parametrize("window", [0, 150])
def test_long_prompts_converted_once_or_in_place(D, ps, dtype, window):
    """More rows than are converted in place: room for all, for the first, or for none of the sequences."""
    rows, lengths = [250, 60, 410], [250, 500, 700]
    outs = []
    for room in (256 << 20, 140000 * (64 if D <= 64 else 128 if D <= 128 else 256) // 128, 0):
        u = Setup4(lengths, 1, D, ps, Hq=16, seed=31, room=room)
        outs.append(check_attend(u, rows, dtype, window).clone())
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("rows,lengths,H,G,D,ps,window", [
    ([20], [3000], 1, 1, 128, 64, 0), ([40, 3], [2000, 700], 1, 4, 64, 16, 0), ([20, 20, 1], [1100, 20, 0], 2, 2, 256, 32, 0),
    ([300], [2000], 1, 1, 256, 128, 500), ([5], [5000], 1, 8, 192, 48, 0), ([70], [4500], 1, 2, 80, 64, 3000),
    ([33], [40], 1, 1, 160, 16, 0)])
def test_prompts_in_parts_and_wide_heads(rows, lengths, H, G, D, ps, window):
    u = Setup4(lengths, H, D, ps, Hq=H * G, seed=29, room=0)
    first = check_attend(u, rows, "bf16", window)
    assert torch.equal(first, check_attend(u, rows, "bf16", window))


PARTS = [     # the long axis is cut: few rows, and prompts of few row tiles
    ([1], [8000], 1, 2, 64, 16, 0), ([1], [20000], 2, 8, 256, 128, 0), ([2, 1], [9000, 17], 1, 4, 128, 64, 0),
    ([4], [6000], 1, 4, 80, 48, 0), ([1], [16000], 1, 4, 128, 64, 12345), ([20], [3000], 1, 1, 128, 64, 0),
    ([300], [2000], 1, 1, 256, 128, 500), ([17], [16000], 2, 2, 128, 128, 0)]
AHEAD = [([250, 60, 410], [250, 500, 700], 1, 16, 128, 64, 0), ([900, 20], [1000, 300], 1, 8, 256, 32, 0)]
WINDOWS = [(rows, lengths, 1, G, 64, 16, w)
           for rows, lengths, G in (([1, 2], [300, 131], 3), ([70, 40], [700, 131], 2))
           for w in (1, 2, 16, 17, 63, 64, 65)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,lengths,H,G,D,ps,window,table", [case + (z,) for case in ATTENDS + PARTS + AHEAD + WINDOWS for z in (
    ("short", "long") if max(case[0]) * case[3] <= 16 else ("short",))])
def test_every_token_counts_once(rows, lengths, H, G, D, ps, window, table, dtype):
    """All scores are equal, and token t's value is 7 scales in element t mod D and 0 elsewhere: an output
    is a count of tokens over another (test_gpu_cache_tokens.py has the tolerance's derivation; the
    weights are 2^0 here)."""
    u = Setup4(lengths, H, D, ps, Hq=H * G, seed=60, v_unit=1.0, width=long_table(lengths, H, ps) if table == "long" else 1)
    kc, ks, vc, vs = u.held(lambda s: np.zeros(s, np.int8), lambda s: np.full(s, 56))       # scales of 1
    for t, n in zip(u.table, lengths):
        at = np.arange(max(n, 0))
        vc[t[at // ps], :, at % ps // 16, at % 16, at % D] = 7
    u.fill(kc, ks, vc, vs)
    u.upload()
    Q = torch.randn((sum(rows), H * G, D), device="cuda").to(TDT[dtype])
    pos = np.concatenate([np.arange(n - r, n) for r, n in zip(rows, lengths)])[:, None]
    lo = np.maximum(pos - window + 1, 0) if window else np.zeros_like(pos)
    d = np.arange(D)[None]
    want = ((pos - d) // D - (lo - 1 - d) // D) * 7 / np.maximum(pos - lo + 1, 1)
    want[pos[:, 0] < 0] = 0.0
    O = torch.full_like(Q, float("nan"))
    u.cache.attend(Q, O, u.len, u.pages, offsets=offsets_of(rows), max_new=max(rows), window=window)
    got = O.double().cpu().numpy()
    off = np.abs(got - want[:, None]) > want[:, None] * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -20)
    assert not (off | np.isnan(got)).any(), f"{off.sum()} of {off.size} off, first {np.argwhere(off | np.isnan(got))[0]}"
    assert u.cache.status() == mlora.MLORA_OK


def test_long_sums_of_fp32_rows_keep_their_bits():
    """Values of one sign over many tokens, single rows and prompts (bounds as in test_gpu_cache.py)."""
    D, ps, n = 64, 64, 16000
    rng = np.random.default_rng(32)
    for B, R in ((304, 1), (152, 20)):
        u = Setup4([n], 1, D, ps, seed=33, spare=0)
        vc, vs = rng.integers(3, 8, (u.n_pages, 1, 4, 16, D)).astype(np.int8), rng.integers(50, 60, (u.n_pages, 1, 4, 16, D // 16))
        kc, ks, _, _ = u.held(lambda s: rng.integers(-7, 8, s).astype(np.int8), lambda s: rng.integers(44, 60, s))
        u.fill(kc, ks, vc, vs)
        u.upload()
        q = torch.from_numpy((rng.standard_normal((B * R, 1, D)) * 0.3).astype(F)).cuda()
        o = torch.full_like(q, float("nan"))
        lengths = torch.full((B,), n, dtype=torch.int32, device="cuda")
        u.cache.attend(q, o, lengths, u.pages.expand(B, -1).contiguous(), offsets=offsets_of([R] * B), max_new=R)
        k, v = (torch.from_numpy(u.values(keys, None, 0)[:, 0]).cuda() for keys in (True, False))
        pos = n - R + torch.arange(B * R, device="cuda") % R
        x = D ** -0.5 * q[:, 0].double() @ k.T
        x = x.masked_fill(torch.arange(n, device="cuda")[None] > pos[:, None], -float("inf"))
        want = torch.softmax(x, dim=1) @ v
        assert (o[:, 0].double() - want).norm() < 2.0 ** -18 * want.norm()
        assert u.cache.status() == mlora.MLORA_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,lengths,G,D,ps", [([150], [2500], 2, 128, 64), ([40, 90], [1500, 800], 1, 64, 64), ([1, 1], [2500, 900], 4, 128, 64)])
def test_scores_that_outgrow_the_bound_at_every_step(rows, lengths, G, D, ps, dtype):
    """Every 64 tokens' scores lie some 13 above the last ones': weights that a step first takes are dropped."""
    u = Setup4(lengths, 1, D, ps, Hq=G, seed=52, k_unit=1.0)
    sign = np.where(np.random.default_rng(53).integers(0, 2, D) > 0, 1, -1).astype(np.int8)
    kc, ks, vc, vs = u.held(lambda s: np.random.default_rng(54).integers(-7, 8, s).astype(np.int8), lambda s: np.full(s, 56))
    kc[:] = 7 * sign
    for t in u.table:
        for j, page in enumerate(t[t >= 0]):
            ks[page] = e4m3_of(np.array([13.0 * (j + 1) / (7 * D ** 0.5)]))[0]
    u.fill(kc, ks, vc, vs)
    u.upload()
    q = np.random.default_rng(55).uniform(0.9, 1.1, (sum(rows), G, D)).astype(F) * sign.astype(F)
    check_attend(u, rows, dtype, q=q)


# ---- steps out of range ---------------------------------------------------- #
def test_out_of_range_steps_are_reported_and_touch_nothing_else():
    u = Setup4([40, 40, 40], 2, 64, 16, Hq=2, seed=21)
    before = u.dev.clone()
    rows = torch.randn((3, 2, 64), device="cuda").bfloat16()
    out = torch.full_like(rows, 3.0)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
    good = dict(lengths=u.len, pages=u.pages, offsets=i32([0, 1, 2, 3]), max_new=1)
    spare = [p for p in range(u.n_pages) if p not in u.table]

    def calls(**kw):
        for max_new in (1, 20):          # (the two forms of append)
            a = {**good, "max_new": max_new, **kw}
            u.cache.append(rows, rows, a["lengths"], a["pages"], offsets=a["offsets"], max_new=a["max_new"])
            u.cache.attend(rows, out, a["lengths"], a["pages"], offsets=a["offsets"], max_new=a["max_new"])
            assert u.cache.status() == mlora.MLORA_ERR_DEVICE_STEP
            assert u.cache.status() == mlora.MLORA_OK     # read and cleared
            assert torch.equal(u.dev[spare], before[spare])

    bad_page = u.pages.clone()
    bad_page[1, 2] = u.n_pages
    calls(pages=bad_page)
    page = int(u.table[1, 2])
    assert torch.equal(u.dev[page], before[page])        # nothing was stored for sequence 1
    bad_page[1, 2] = -1
    calls(pages=bad_page)
    calls(lengths=i32([40, 49, 40]))                           # more than the table holds
    calls(lengths=i32([40, -3, 40]))
    assert torch.all(out[1] == 0)
    out.fill_(3.0)
    calls(offsets=i32([0, 1, 7, 3]))                           # past T, then decreasing
    assert torch.all(out[1:] == 3.0)
    calls(offsets=i32([0, 0, 0, 3]), max_new=1)                # more rows than max_new


@pytest.mark.parametrize("rows", [1, 20])
def test_tokens_of_a_bad_page_read_as_zero(rows):
    u = Setup4([64, 20], 1, 64, 16, Hq=2, seed=22)
    keep = u.table.copy()
    u.table[0, 1] = u.n_pages + 5
    u.pages = torch.from_numpy(u.table).cuda()
    q = torch.randn((2 * rows, 2, 64), device="cuda")
    o = torch.empty_like(q)
    u.cache.attend(q, o, u.len, u.pages, offsets=offsets_of([rows, rows]), max_new=rows)
    k = torch.empty((64, 1, 64), device="cuda")
    v = torch.empty_like(k)
    u.cache.read(k, v, u.len[:1], u.pages[:1], offsets=offsets_of([64]), max_new=64)
    assert u.cache.status() == mlora.MLORA_ERR_DEVICE_STEP
    assert not k[16:32].any() and k[48:].any() and not v[16:32].any()
    for t in range(24, 28):      # and through the form for few rows
        u.cache.read(k[:1], v[:1], torch.tensor([t + 1], dtype=torch.int32, device="cuda"), u.pages[:1])
        assert not k[:1].any() and not v[:1].any()
    u.table = keep
    kc, ks, vc, vs = (x for keys in (True, False) for x in unpack(u.blocks, keys))
    ks[keep[0, 1]] = vs[keep[0, 1]] = 0
    u.fill(kc, ks, vc, vs)
    want, A, S = plain_attend(u, as_np(q), [rows, rows], 0.125, 0)
    assert (np.abs(as_np(o) - want) <= tolerance(want, A, S, "f32")).all()


def test_refusals():
    u = Setup4([20, 5], 2, 64, 16, Hq=4, seed=23)
    k = torch.zeros((2, 2, 64), device="cuda", dtype=torch.bfloat16)
    q = torch.zeros((2, 4, 64), device="cuda", dtype=torch.bfloat16)
    for bad in (lambda: u.cache.append(k, k.float(), u.len, u.pages),
                lambda: u.cache.append(k.half(), k.half(), u.len, u.pages),
                lambda: u.cache.append(q, q, u.len, u.pages),
                lambda: u.cache.attend(k, k, u.len, u.pages),
                lambda: u.cache.append(k.cpu(), k.cpu(), u.len, u.pages),
                lambda: Cache4(u.dev.char(), 4),
                lambda: Cache4(u.dev[..., 1:], 4),
                lambda: Cache4(u.dev.transpose(0, 1), 4),
                lambda: Cache4(u.dev[0], 4),
                lambda: Cache4(u.dev.cpu(), 4)):
        with pytest.raises(ValueError):
            bad()
    odd = torch.zeros(u.dev.numel() + 8, dtype=torch.uint8, device="cuda")[8:].view(u.dev.shape)
    for bad, status in ((lambda: u.cache.attend(q, q.clone(), u.len, u.pages, window=-1), mlora.MLORA_ERR_INVALID_ARG),
                        (lambda: u.cache.append(k, k, u.len, u.pages, max_new=-1), mlora.MLORA_ERR_INVALID_ARG),
                        (lambda: Cache4(u.dev, 3), mlora.MLORA_ERR_INVALID_ARG),
                        (lambda: Cache4(u.dev, 4, k_unit=0.0), mlora.MLORA_ERR_INVALID_ARG),
                        (lambda: Cache4(u.dev, 4, v_unit=float("nan")), mlora.MLORA_ERR_INVALID_ARG),
                        (lambda: Cache4(odd, 4), mlora.MLORA_ERR_INVALID_ARG),
                        (lambda: u.cache.attend(q, q.clone(), u.len, u.pages, scale=2e-37), mlora.MLORA_ERR_UNSUPPORTED)):
        with pytest.raises(mlora.MloraError) as e:
            bad()
        assert e.value.status == status


def test_empty_steps_do_nothing():
    u = Setup4([20], 2, 64, 16, seed=24)
    none = torch.zeros((0, 2, 64), device="cuda")
    before = u.dev.clone()
    u.cache.append(none, none, u.len[:0], u.pages[:0])
    u.cache.read(none, none, u.len[:0], u.pages[:0])
    u.cache.attend(none, none, u.len[:0], u.pages[:0])
    u.cache.append(none, none, u.len, u.pages, offsets=offsets_of([0]), max_new=0)
    u.cache.attend(none, none, u.len, u.pages, offsets=offsets_of([0]), max_new=4)
    assert torch.equal(u.dev, before) and u.cache.status() == mlora.MLORA_OK


# ---- streams, graphs, large offsets ---------------------------------------- #
@pytest.mark.parametrize("n", [1, 40])
def test_a_step_on_another_stream_and_in_a_graph(n):
    u = Setup4([100, 50], 2, 128, 16, Hq=4, seed=25)
    rng = np.random.default_rng(26)
    K, V = (strided(rng.standard_normal((2 * n, 2, 128)).astype(F), "bf16") for _ in range(2))
    Q = strided(rng.standard_normal((2 * n, 4, 128)).astype(F), "bf16")
    want = torch.empty_like(Q)
    step = dict(offsets=offsets_of([n, n]), max_new=n)
    u.cache.append(K, V, u.len, u.pages, **step)
    u.cache.attend(Q, want, u.len, u.pages, **step)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = torch.zeros_like(Q)
    side.wait_stream(torch.cuda.current_stream())
    u.cache.append(K, V, u.len, u.pages, **step, stream=side)
    u.cache.attend(Q, got, u.len, u.pages, **step, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        u.cache.append(K, V, u.len, u.pages, **step)
        u.cache.attend(Q, got, u.len, u.pages, **step)
    for _ in range(2):
        got.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    assert u.cache.status(side) == mlora.MLORA_OK


@pytest.mark.parametrize("R", [1, 30])
def test_blocks_past_32_bit_offsets(R):
    """Blocks past 2^32 bytes of the array (4.8 GB)."""
    H, ps, D, n_pages = 4, 128, 128, 65600
    blocks = torch.empty((n_pages, H, ps // 16, 18 * D), dtype=torch.uint8, device="cuda")
    blocks[[0, 40000, 65590, 65599]] = 0xFF
    cache = Cache4(blocks, 8)
    table = torch.tensor([[65599, 40000], [0, 65590]], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    K, V = (torch.randn((400, H, D), device="cuda", generator=g) for _ in range(2))
    length = torch.tensor([200, 200], dtype=torch.int32, device="cuda")
    cache.append(K, V, length, table, offsets=offsets_of([200, 200]), max_new=200)
    rk, rv = torch.empty_like(K), torch.empty_like(V)
    cache.read(rk, rv, length, table, offsets=offsets_of([200, 200]), max_new=200)
    # a code is off by half a step, of at most 1/7 + 1/16 of it of the group's largest value (some 4.5 here)
    assert (rk - K).abs().max() <= 0.5 * 1.07 / 7 * K.abs().max() and (rv - V).abs().max() <= 0.5 * 1.07 / 7 * V.abs().max()
    Q = torch.randn((2 * R, 8, D), device="cuda", generator=g)
    O = torch.empty_like(Q)
    cache.attend(Q, O, length, table, offsets=offsets_of([R, R]), max_new=R)
    for b in range(2):
        k, v = (x[200 * b:200 * b + 200].double().repeat_interleave(2, dim=1) for x in (rk, rv))
        for i in range(R):
            n = 200 - R + i + 1
            w = torch.einsum("hd,thd->ht", Q[b * R + i].double(), k[:n]) * D ** -0.5
            want = torch.einsum("ht,thd->hd", w.softmax(-1), v[:n])
            assert (O[b * R + i] - want).abs().max() < 1e-3 * want.abs().max()
    assert cache.status() == mlora.MLORA_OK


@pytest.mark.parametrize("length", [700, 2 ** 30])
def test_append_and_read_launched_for_2_31_rows(length):
    """Five rows of a step that may hold 2^31 - 1 (one row of memory), at the end of a sequence."""
    ps, D, T = 256, 16, 2 ** 31 - 1
    table = torch.full((1, 2 ** 30 // ps), -1, dtype=torch.int32, device="cuda")   # (one block is touched)
    table[0, (length - 1) // ps] = 1
    blocks = torch.zeros((3, 1, ps // 16, 18 * D), dtype=torch.uint8, device="cuda")
    cache = Cache4(blocks, 1)
    row = torch.randn((1, 1, D), device="cuda")
    step = dict(lengths=torch.tensor([length], dtype=torch.int32, device="cuda"), pages=table, offsets=offsets_of([5]))
    K = row.expand(T, 1, D)
    cache.append(K, K, **step, max_new=T)
    held = blocks.cpu().numpy()
    codes, scales = unpack(held, True)
    want = quantised(as_np(row)[0, 0], 0.0625)
    for p in range(length - 5, length):
        at = (1, 0, p % ps // 16, p % 16)
        np.testing.assert_array_equal(codes[at], want[0])
        assert scales[at] == want[1][0]
    assert np.count_nonzero(scales) == 5 and np.count_nonzero(unpack(held, False)[1]) == 5
    back = torch.full_like(row, 7.0)
    cache.read(back.expand(T, 1, D), back.expand(T, 1, D), **step, max_new=T)   # (five equal rows into one)
    np.testing.assert_array_equal(as_np(back)[0, 0], want[0] * E4M3[want[1][0]].astype(F) * F(0.0625))
    assert cache.status() == mlora.MLORA_OK


@pytest.mark.parametrize("rows,dtype,off", [(1, "bf16", 2.0 ** -7), (1, "f32", 2.0 ** -7), (20, "bf16", 0.06), (20, "f32", 2.0 ** -7)])
@pytest.mark.parametrize("D", [64, 256])
def test_attention_over_2_30_tokens(rows, dtype, off, D):
    """Blocks that are all one page, under equal weights: the mean of its values (test_gpu_cache_edges.py has
    the bounds)."""
    ps, L = 256, 2 ** 30
    u = Setup4([2 * ps], 1, D, ps, seed=50, spare=0)
    _, _, vc, vs = u.held(lambda s: np.random.default_rng(51).integers(3, 8, s).astype(np.int8), lambda s: np.full(s, 56))
    u.fill(vc, vs, vc, vs)
    u.upload()
    page = int(u.table[0, 0])
    table = torch.full((1, L // ps), page, dtype=torch.int32, device="cuda")
    Q = torch.zeros((rows, 1, D), dtype=TDT[dtype], device="cuda")
    O = torch.full_like(Q, float("nan"))
    u.cache.attend(Q, O, torch.tensor([L], dtype=torch.int32, device="cuda"), table, offsets=offsets_of([rows]), max_new=rows)
    want = torch.from_numpy(u.values(False, None, 0)[:ps, 0].mean(0)).cuda()
    assert ((O[:, 0].double() - want).abs() <= off * want).all()
    assert u.cache.status() == mlora.MLORA_OK


@pytest.mark.parametrize("rows", [1, 20])
def test_an_expired_wait_is_reported_until_read(rows):
    """As over 8 bits: a wait that gives up sets the status; later calls leave it set and are right."""
    u = Setup4([300, 20], 1, 64, 16, Hq=2, seed=56)
    q = strided(np.random.default_rng(57).standard_normal((2 * rows, 2, 64)).astype(F), "bf16")
    out = [torch.empty_like(q) for _ in range(2)]
    step = dict(offsets=offsets_of([rows, rows]), max_new=rows)
    u.cache.attend(q, out[0], u.len, u.pages, **step)
    assert u.cache.status() == mlora.MLORA_OK
    mlora.mlora_debug_cache_expire_wait(u.cache.handle, 2_000_000, torch.cuda.current_stream().cuda_stream)
    u.cache.attend(q, out[1], u.len, u.pages, **step)
    assert u.cache.status() == mlora.MLORA_ERR_DEVICE_TIMEOUT
    assert u.cache.status() == mlora.MLORA_OK
    assert torch.equal(out[0], out[1])
