"""Attention over the caches where scores are large: finite queries and keys give the softmax of
their scores, as far as fp32 holds these."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():   # pragma: no cover - CPU machine
    pytest.skip("needs a GPU", allow_module_level=True)

from heterogeneous_lora_gemm_gb300 import mlora  # noqa: E402
from test_gpu_cache import F, Setup, TDT, offsets_of  # noqa: E402
from test_gpu_cache4 import Setup4  # noqa: E402

# rows, lengths, key heads, query heads of each, head size, page, columns of the page table: every form of the kernels
FEW = [([1], [300], 2, 4, 128, 64, 1), ([1], [300], 2, 4, 128, 64, 3000), ([1], [9000], 1, 8, 64, 16, 1), ([1, 1], [70, 300], 2, 4, 48, 32, 1),
       ([4], [600], 1, 4, 128, 48, 1), ([3, 2], [300, 290], 1, 3, 96, 16, 1), ([1], [700], 1, 2, 256, 32, 1), ([9], [400], 1, 1, 256, 64, 1)]
MANY = [([40], [300], 1, 2, 128, 64, 1), ([20], [3000], 1, 1, 128, 64, 1), ([150, 30], [500, 300], 1, 2, 64, 16, 1), ([40], [300], 1, 1, 256, 64, 1),
        ([250, 60], [1250, 500], 1, 16, 128, 64, 1), ([900], [1300], 1, 8, 80, 32, 1)]


def attended(u, q, rows, scale, dtype):
    Q = torch.from_numpy(np.array(q, F, order="C")).cuda().to(TDT[dtype])
    assert np.array_equal(Q.float().cpu().numpy(), q)
    O = torch.full_like(Q, float("nan"))
    u.cache.attend(Q, O, u.len, u.pages, offsets=offsets_of(rows), max_new=max(rows), scale=scale)
    assert u.cache.status() == mlora.MLORA_OK
    return O.double().cpu().numpy()


@pytest.mark.parametrize("rows,lengths,H,G,D,ps,width", FEW + MANY)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("negative,at", [(False, "first"), (True, "last")])
def test_one_token_with_all_of_the_weight(rows, lengths, H, G, D, ps, width, dtype, bits, negative, at):
    """One token's score lies a seventh above all others', of which 2^-10000 of the weight is left at the
    least: the output is that token's value, whose rounding (and the quotient's, and over 8 bits the product's
    with its scale) is all that is off."""
    if bits == 4:
        u = Setup4(lengths, H, D, ps, Hq=H * G, seed=90, k_unit=1.0, v_unit=0.5, width=width)
        kc, ks, vc, vs = u.held(lambda s: np.random.default_rng(91).integers(-7, 8, s).astype(np.int8), lambda s: np.full(s, 56))
        most = 7
    else:
        u = Setup(lengths, H, D, ps, Hq=H * G, seed=90)
        kc, most = u.kc, 126
        u.ks[np.isfinite(u.ks)] = 1.0 / 18.0
    sign = np.where(np.random.default_rng(92).integers(0, 2, D) > 0, 1, -1).astype(np.int8)
    tokens = [3 if at == "first" else n - r for n, r in zip(lengths, rows)]      # (every row sees it)
    kc[:] = (-most if negative else most // 7 * 6) * sign
    for b, t in enumerate(tokens):
        place = (u.table[b, t // ps], slice(None)) + ((t % ps // 16, t % 16) if bits == 4 else (t % ps,))
        kc[place] = (-most // 7 * 6 if negative else most) * sign
    if bits == 4:
        u.fill(kc, ks, vc, vs)
    u.upload()
    for log2_score in (18, 23, 25, 28, 31, 33, 40, 100):
        a = log2_score - int(np.ceil(np.log2(D)))               # scores of 7 D 2^a scale
        scale, q = (2.0 ** -3, 2.0 ** a) if a <= 60 else (2.0 ** (a - 63), 2.0 ** 60)
        got = attended(u, np.broadcast_to(sign * q, (sum(rows), H * G, D)), rows, scale, dtype)
        for b, t in enumerate(tokens):
            v = (u.values(False, None, b) if bits == 4 else u.values(u.vc, u.vs, b))[t][:, None]   # [H, 1, D]
            mine = got[sum(rows[:b]):sum(rows[:b + 1])].reshape(rows[b], H, G, D)
            bad = ~(np.abs(mine - v) <= (2.0 ** -8 if dtype == "bf16" else 2.0 ** -20) * np.abs(v))
            assert not bad.any(), f"2^{log2_score}: {bad.sum()} of {bad.size} off, first {np.argwhere(bad)[0]}: {mine[bad][:3]}"


@pytest.mark.parametrize("rows,lengths,H,G,D,ps,width", FEW + MANY)
@pytest.mark.parametrize("order", ["rising", "mixed"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_neighbouring_scores_of_any_size(rows, lengths, H, G, D, ps, width, order, dtype):
    """Scores that are whole numbers N + d, d in 0 .. 7 beside N of up to 23 bits, so that fp32 holds each
    exactly, under factors that make a difference of 1 a power of up to 2^30: the weights are those of the d's.
    Tolerance: in fp32 the differences are exact but for the factor's two roundings, and the weights of powers
    down to 2^-40 are off by 2^-24 * 3 * 40 of themselves and the exponential's 2^-22, both of numerator and denominator:
    2^-16.  bf16: the weights round to 8 bits at the least, the output once (and 2^-37 as in test_gpu_cache4.py)."""
    u = Setup4(lengths, H, D, ps, Hq=H * G, seed=93, k_unit=1.0, v_unit=0.5, width=width)
    rng = np.random.default_rng(94)
    kc, ks, vc, vs = u.held(lambda s: rng.integers(-7, 8, s).astype(np.int8), lambda s: np.full(s, 56))
    kc[..., 16:], kc[..., :16] = 7, 0
    step = [np.arange(n) * 8 // n if order == "rising" else rng.integers(0, 8, n) for n in lengths]
    for t, d in zip(u.table, step):
        at = np.arange(d.size)
        kc[t[at // ps], :, at % ps // 16, at % 16, 0] = d[:, None]
    u.fill(kc, ks, vc, vs)
    u.upload()
    for log2_common, log2_step in ((10, 0.1), (20, 0.3), (21, 1.3), (22, 0.4), (22, 7.1), (22, 30.0), (23, 2.9), (23, 17.6)):
        q = np.full(D, 2.0 ** (log2_common - int(np.log2((D - 16) * 7))))
        q[:16] = 1.0
        scale = float(F(log2_step * np.log(2.0)))
        got = attended(u, np.broadcast_to(q, (sum(rows), H * G, D)), rows, scale, dtype)
        for b, (n, length) in enumerate(zip(rows, lengths)):
            v = u.values(False, None, b)
            low = 2.0 ** -37 * length * np.abs(v).max()
            for i in range(n):
                seen = length - n + i + 1
                p = np.exp(scale * (step[b][:seen] - step[b][:seen].max()))
                p /= p.sum()
                want, A = (np.tensordot(p, x[:seen], 1)[:, None] for x in (v, np.abs(v)))
                mine = got[sum(rows[:b]) + i].reshape(H, G, D)
                off = 2.0 ** -8 * np.abs(want) + 2.0 ** -7 * A if dtype == "bf16" else 2.0 ** -16 * A
                bad = ~(np.abs(mine - want) <= off + low)
                assert not bad.any(), (f"2^{log2_common} by 2^{log2_step}, row {i} of {b}: {bad.sum()} of {bad.size} off, "
                                       f"first {np.argwhere(bad)[0]}: {mine[bad][:3]}")


@pytest.mark.parametrize("rows,lengths,G,D", [([3], [1], 2, 128), ([4, 1], [2, 300], 4, 64), ([9], [3], 1, 256), ([40], [7], 2, 128),
                                              ([200, 150], [60, 400], 1, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [8, 4])
def test_rows_that_see_no_token_are_zeros_whatever_their_queries(rows, lengths, G, D, dtype, bits):
    """Rows at negative positions beside rows that see something; the others are as without them."""
    u = (Setup4 if bits == 4 else Setup)(lengths, 1, D, 64, Hq=G, seed=95)
    q = torch.randn((sum(rows), G, D), device="cuda").to(TDT[dtype])
    out = []
    pos = np.concatenate([np.arange(n - r, n) for r, n in zip(rows, lengths)])
    blind = torch.from_numpy(pos < 0).cuda()
    for bad in (1.0, float("nan"), float("inf"), -float("inf")):
        Q = q.clone()
        Q[blind, :, 5] = bad
        O = torch.full_like(Q, 9.0)
        u.cache.attend(Q, O, u.len, u.pages, offsets=offsets_of(rows), max_new=max(rows))
        out.append(O)
        assert torch.all(O[blind] == 0) and torch.equal(O, out[0])
    assert u.cache.status() == mlora.MLORA_OK
