"""The 8-bit cache's attention at the edges of what its calls accept: against 64 bits, with the
tolerances of test_gpu_cache.py unless a test says otherwise."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():   # pragma: no cover - CPU machine
    pytest.skip("needs a GPU", allow_module_level=True)

from heterogeneous_lora_gemm_gb300 import Cache, mlora  # noqa: E402
from test_gpu_cache import F, Setup, as_np, check_attend, offsets_of, plain_attend, strided, tolerance  # noqa: E402


# ---- windows --------------------------------------------------------------- #
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,lengths,H,G,D,ps", [
    ([7, 1, 6], [3, 90, 2], 2, 2, 64, 16),                # few rows, some at negative positions
    ([5, 3], [2, 700], 1, 1, 256, 32),
    ([6, 40], [2, 30], 2, 4, 128, 64),                    # prompts, left-padded
    ([300, 20], [7, 500], 1, 16, 128, 64),                # and converted ahead
])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 8, 2 ** 30])
def test_a_window_larger_than_any_position_is_no_window(rows, lengths, H, G, D, ps, window, dtype):
    u = Setup(lengths, H, D, ps, Hq=H * G, seed=40)
    limited = check_attend(u, rows, dtype, window)
    assert torch.equal(limited, check_attend(u, rows, dtype, 0))


# ---- value scales far below 1 ------------------------------------------------ #
# rows, lengths, H, G, D, page, bytes for prompts (few rows; prompts in place; prompts converted ahead)
TINY = [([1, 1], [520, 64], 1, 2, 64, 16, 0), ([130], [450], 1, 2, 64, 16, 0), ([70, 20], [300, 90], 1, 3, 128, 64, 0),
        ([40], [400], 1, 2, 256, 32, 0), ([250, 60], [250, 500], 1, 16, 128, 64, 256 << 20)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tiny", [2.0 ** -63, 2.0 ** -65, 2.0 ** -119, 1e-36, 1e-38, 1e-41])
@pytest.mark.parametrize("rows,lengths,H,G,D,ps,room", TINY)
def test_tokens_of_tiny_value_blocks_keep_their_weight(rows, lengths, H, G, D, ps, room, tiny, dtype):
    """Every other block's values are next to nothing; its tokens' weights stay in the softmax's sum."""
    u = Setup(lengths, H, D, ps, Hq=H * G, seed=41)
    for t in u.table:
        u.vs[t[1::2][t[1::2] >= 0]] = tiny
    u.upload()
    u.cache = Cache(*u.dev, H * G, prompt_bytes=room)
    check_attend(u, rows, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,lengths,H,G,D,ps,room", TINY)
def test_values_that_are_all_tiny(rows, lengths, H, G, D, ps, room, dtype):
    """Value scales around 2^-96: attention of values times 2^90 would give the outputs times 2^90."""
    u = Setup(lengths, H, D, ps, Hq=H * G, seed=42, v_size=0.7 * 2.0 ** -90)
    u.cache = Cache(*u.dev, H * G, prompt_bytes=room)
    Q = strided(np.random.default_rng(43).standard_normal((sum(rows), H * G, D)).astype(F), dtype)
    O = torch.empty_like(Q)
    u.cache.attend(Q, O, u.len, u.pages, offsets=offsets_of(rows), max_new=max(rows))
    o, A, S = (x * 2.0 ** 90 if k < 2 else x for k, x in enumerate(plain_attend(u, as_np(Q), rows, D ** -0.5, 0)))
    got = O.double().cpu().numpy() * 2.0 ** 90
    assert (np.abs(got - o) <= tolerance(o, A, S, dtype)).all()
    assert u.cache.status() == mlora.MLORA_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 40])
def test_a_block_of_denormal_rows_beside_normal_ones(rows, dtype):
    """As the append stores it: a scale of some 1e-40 and codes of 0."""
    u = Setup([96], 1, 64, 32, Hq=2, seed=44)
    x = np.random.default_rng(45).standard_normal((96, 1, 64)).astype(F)
    x[32:64] *= F(1e-38)
    K = strided(x, dtype)
    u.cache.append(K, K, u.len, u.pages, offsets=offsets_of([96]), max_new=96)
    u.kc, u.ks, u.vc, u.vs = (t.cpu().numpy() for t in u.dev)
    assert 0 < u.vs[u.table[0, 1], 0] < 1e-39 and not u.vc[u.table[0, 1]].any()
    check_attend(u, [rows], dtype)


# ---- creation --------------------------------------------------------------------- #
@pytest.mark.parametrize("rows,lengths,G", [([1, 1], [3000, 2500], 4), ([30], [2500], 4)])
def test_a_new_cache_may_be_used_on_any_stream_at_once(rows, lengths, G):
    """Its workspace is cleared when the call returns, however much is queued on the default stream:
    attention split over many CTAs (their arrivals are counted in it) on a stream that waits for none."""
    u = Setup(lengths, 1, 128, 64, Hq=G, seed=47)
    Q = strided(np.random.default_rng(48).standard_normal((sum(rows), G, 128)).astype(F), "bf16")
    want, off = torch.empty_like(Q), offsets_of(rows)
    u.cache.attend(Q, want, u.len, u.pages, offsets=off, max_new=max(rows))
    side = torch.cuda.Stream()
    got = [torch.zeros_like(Q) for _ in range(4)]
    torch.cuda.synchronize()
    for o in got:
        torch.cuda._sleep(20_000_000)       # some 10 ms on the default stream
        cache = Cache(*u.dev, G)
        assert torch.cuda.default_stream().query()
        cache.attend(Q, o, u.len, u.pages, offsets=off, max_new=max(rows), stream=side)
        assert cache.status(side) == mlora.MLORA_OK
    assert all(torch.equal(o, want) for o in got)


@pytest.mark.parametrize("what", ["cache", "pool"])
def test_a_creation_that_fails_leaves_the_next_calls_alone(what):
    """Out of memory is the answer to that call, and not to the next launch."""
    u = Setup([20], 1, 64, 16, seed=46)
    with pytest.raises(mlora.MloraError) as e:
        if what == "cache":    # a workspace for 2^30 tokens of 256 elements: over a terabyte
            mlora.mlora_cache_create(*[t.data_ptr() for t in u.dev], 1 << 26, 16, 1, 256, 1, 1 << 62)
        else:                  # 2^20 rank units of 2^20 elements: two
            mlora.mlora_pool_create(1, 1 << 20, 16, 1 << 20, 64, mlora.MLORA_BF16, 16)
    assert e.value.status == mlora.MLORA_ERR_OOM
    check_attend(u, [1], "bf16")


# ---- pages that no row sees any more ------------------------------------------ #
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("left", ["none", "not a number"])
@pytest.mark.parametrize("rows,lengths,H,G,D,ps,window,room", [
    ([1, 1, 1], [300, 64, 65], 2, 2, 96, 16, 40, 0),           # 16 tokens of a copied 32 lie behind the window
    ([1, 3], [1000, 700], 1, 4, 128, 32, 100, 0),
    ([1], [5000], 1, 3, 256, 16, 1000, 0),
    ([150, 20], [400, 300], 2, 3, 80, 32, 100, 0),             # prompts: 32 or more of 128
    ([40], [700], 1, 2, 128, 64, 130, 0),
    ([300], [2000], 1, 1, 256, 16, 500, 0),
    ([20], [1500], 1, 4, 64, 48, 77, 0),
    ([250, 60], [2250, 500], 1, 16, 128, 64, 150, 256 << 20),  # and converted ahead
])
def test_pages_behind_the_window_are_not_read(rows, lengths, H, G, D, ps, window, room, left, dtype):
    """Their entries in the page table hold no page, or one with scales that are not numbers."""
    u = Setup(lengths, H, D, ps, Hq=H * G, seed=51)
    free = next(p for p in range(u.n_pages) if p not in u.table)
    assert np.isnan(u.vs[free]).all()
    for t, n, length in zip(u.table, rows, lengths):
        t[:max(0, length - n - window + 1) // ps] = -1 if left == "none" else free
    assert (u.table == (-1 if left == "none" else free)).sum() > 2
    u.upload()
    u.cache = Cache(*u.dev, H * G, prompt_bytes=room)
    check_attend(u, rows, dtype, window)


# ---- sizes near 2^31 -------------------------------------------------------------- #
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("length", [700, 2 ** 30])
def test_append_and_read_launched_for_2_31_rows(length, dtype):
    """Five rows of a step that may hold 2^31 - 1 (one row of memory), at the end of a sequence."""
    ps, D, T = 256, 16, 2 ** 31 - 1
    table = torch.full((1, 2 ** 30 // ps), -1, dtype=torch.int32, device="cuda")   # (one block is touched)
    table[0, (length - 1) // ps] = 1
    shape = (3, 1, ps, D)
    pages = [torch.zeros(shape, dtype=torch.int8, device="cuda"), torch.zeros(shape[:2], device="cuda")]
    pages += [t.clone() for t in pages]
    cache = Cache(*pages, 1)
    row = strided(np.random.default_rng(49).standard_normal((1, 1, D)).astype(F), dtype)
    step = dict(lengths=torch.tensor([length], dtype=torch.int32, device="cuda"), pages=table, offsets=offsets_of([5]))
    K = row.expand(T, 1, D)
    cache.append(K, K, **step, max_new=T)
    place = slice((length - 5) % ps, (length - 5) % ps + 5)
    q = torch.clamp(torch.round(row[0, 0].float() / (row.float().abs().max() / 127)), -127, 127)
    for codes, scale in ((pages[0], pages[1]), (pages[2], pages[3])):
        assert torch.equal(codes[1, 0, place].float(), q.expand(5, D))
        assert torch.count_nonzero(codes) == 5 * torch.count_nonzero(q) and torch.count_nonzero(scale) == 1
    back = torch.full_like(row, 7.0)
    cache.read(back.expand(T, 1, D), back.expand(T, 1, D), **step, max_new=T)   # (five equal rows into one)
    assert torch.equal(back[0, 0], (q * pages[1][1]).to(back.dtype))
    assert cache.status() == mlora.MLORA_OK


def test_attention_of_more_row_tiles_than_32_bits_count_is_refused():
    shape = (2, 1025, 16, 16)
    pages = [torch.zeros(shape, dtype=torch.int8, device="cuda"), torch.zeros(shape[:2], device="cuda")]
    cache = Cache(*pages, *pages, 1025)
    Q = torch.zeros((1, 1, 16), device="cuda").expand(2 ** 30, 1025, 16)
    with pytest.raises(mlora.MloraError) as e:
        cache.attend(Q, Q, torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                     offsets=offsets_of([1]), max_new=2 ** 30)
    assert e.value.status == mlora.MLORA_ERR_UNSUPPORTED


@pytest.mark.parametrize("rows,dtype,off", [(1, "bf16", 2.0 ** -7), (1, "f32", 2.0 ** -7), (20, "bf16", 0.06), (20, "f32", 2.0 ** -7)])
@pytest.mark.parametrize("D", [64, 256])
def test_attention_over_2_30_tokens(rows, dtype, off, D):
    """Blocks that are all one page, under equal weights: the mean of its values.  At the most 2^30 / 152
    tokens are summed in one place.  The tensor cores cut sums off at every 16 tokens: 2^-23 of the sum so
    far at 441000 of them for prompts of bf16 rows, 5.3%; single tokens' sums are a twelfth as long
    (2^30 / (304 x 4) tokens: 55000 times, 0.7%), and fp32 rows' are taken out of the tensor cores."""
    ps, L = 256, 2 ** 30
    rng = np.random.default_rng(50)
    codes = torch.from_numpy(rng.integers(60, 128, (2, 1, ps, D)).astype(np.int8)).cuda()
    scale = torch.full((2, 1), 2.0 ** -7, device="cuda")
    cache = Cache(codes, scale, codes, scale, 1)
    table = torch.ones((1, L // ps), dtype=torch.int32, device="cuda")
    Q = torch.zeros((rows, 1, D), dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device="cuda")
    O = torch.full_like(Q, float("nan"))
    cache.attend(Q, O, torch.tensor([L], dtype=torch.int32, device="cuda"), table, offsets=offsets_of([rows]), max_new=rows)
    want = codes[1, 0].double().mean(0) * 2.0 ** -7
    assert ((O[:, 0].double() - want).abs() <= off * want).all()
    assert cache.status() == mlora.MLORA_OK


# ---- bounds that move at every step --------------------------------------------------- #
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,lengths,G,D,ps", [([150], [2500], 2, 128, 64), ([40, 90], [1500, 800], 1, 64, 64),
                                                 ([140], [1000], 2, 96, 16), ([1, 1], [2500, 900], 4, 128, 64)])
def test_scores_that_outgrow_the_bound_at_every_step(rows, lengths, G, D, ps, dtype):
    """Block after block whose scores lie some 13 above the last one's: the weights that a step first
    takes are of up to 2^19 and more, and dropped."""
    u = Setup(lengths, 1, D, ps, Hq=G, seed=52)
    sign = np.where(np.random.default_rng(53).integers(0, 2, D) > 0, 1, -1)
    u.kc = (sign * np.random.default_rng(54).integers(115, 128, u.kc.shape)).astype(np.int8)
    for t in u.table:
        for j, page in enumerate(t[t >= 0]):
            u.ks[page] = 13.0 * (j + 1) / (121 * D ** 0.5)
    u.upload()
    q = np.random.default_rng(55).uniform(0.9, 1.1, (sum(rows), G, D)).astype(F) * sign.astype(F)
    check_attend(u, rows, dtype, q=q)


# ---- waits that run out ------------------------------------------------------------------ #
def test_an_expired_wait_is_reported_until_read():
    """A pipeline wait that gives up (one that nothing completes, bounded to about a millisecond) sets
    the cache's status; later calls leave it set and are right, the status call reports and clears it."""
    u = Setup([300, 17], 1, 64, 16, Hq=2, seed=56)
    stream = torch.cuda.current_stream().cuda_stream
    assert u.cache.status() == mlora.MLORA_OK
    mlora.mlora_debug_cache_expire_wait(u.cache.handle, 2_000_000, stream)
    Q = strided(np.random.default_rng(57).standard_normal((2, 2, 64)).astype(F), "bf16")
    O = torch.empty_like(Q)
    u.cache.attend(Q, O, u.len, u.pages)
    assert u.cache.status() == mlora.MLORA_ERR_DEVICE_TIMEOUT
    assert u.cache.status() == mlora.MLORA_OK
    assert torch.equal(O, check_attend(u, [1, 1], "bf16", q=as_np(Q)))
    for cycles in (0, 2 ** 31 + 1):
        with pytest.raises(mlora.MloraError) as e:
            mlora.mlora_debug_cache_expire_wait(u.cache.handle, cycles, stream)
        assert e.value.status == mlora.MLORA_ERR_INVALID_ARG


# ---- queries near the end of fp32 ---------------------------------------------------------- #
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,lengths,D", [([1, 1], [300, 64], 128), ([131, 30], [200, 30], 128), ([40], [90], 64), ([20], [90], 256)])
@pytest.mark.parametrize("scale", [0.1, 3.0, 1000.0])
def test_the_largest_queries(rows, lengths, D, scale, dtype):
    """Rows up to 2^128 beside rows of 2^100, and keys that bring the scores of the first to about 1."""
    u = Setup(lengths, 1, D, 64, Hq=2, seed=58)
    u.ks = np.where(np.isnan(u.ks), u.ks, F(2.0 ** -126 / scale / D ** 0.5 / 8) * (1 + u.ks)).astype(F)
    u.upload()
    q = np.random.default_rng(59).uniform(-2.0 ** 100, 2.0 ** 100, (sum(rows), 2, D))
    q[::2] *= 2.0 ** 27.5
    check_attend(u, rows, dtype, q=q.astype(F), scale=scale)
